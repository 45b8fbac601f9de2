// linear_chain.h -- products of many tiles whose epilogues need no LDS: a cross entropy's logits, reduced to their rows'
// statistics or turned into its gradient, and its weights' gradient.
//
// The large tiles' pipeline (linear_fast.h), with a workgroup's tiles as one run of steps: the loads of a tile's last two
// steps are the next tile's first two, which land while this tile's sums pass through the epilogue in registers.  A
// workgroup per tile instead begins every tile with an empty pipeline, all CUs at once: 4096 x 50021 of 256 terms took 181
// us that way and takes 155 now (12.6 a tile, the epilogue 4.4 of it), of 4096 terms 1248 and 1192.
#pragma once

#include "linear_fast.h"
#include "loss_tile.h"

namespace miconv {

// One wave's FM x FN blocks into rows of y in the tensors' type, 16 bytes a lane.
template <class Out, class Block, int FM, int FN>
__device__ __forceinline__ void store_wave(Out* y, int64_t ld, int rows, int columns, const Block (&acc)[FM][FN], int m0, int j0, int lane)
{
    if constexpr (sizeof(Block) == sizeof(f32x16)) {
        // 32 x 32: four columns a quarter
#pragma unroll
        for (int i = 0; i < FM; ++i) {
            const int m = m0 + 32 * i + (lane & 31);
            if (m >= rows) continue;
#pragma unroll
            for (int j = 0; j < FN; ++j)
#pragma unroll
                for (int q = 0; q < 4; ++q) {
                    const int n = j0 + 32 * j + 8 * q + 4 * (lane >> 5);
                    const f32x4 v = {acc[i][j][4 * q], acc[i][j][4 * q + 1], acc[i][j][4 * q + 2], acc[i][j][4 * q + 3]};
                    Out* to = y + m * ld + n;
                    if (n + 4 <= columns) {
                        __builtin_memcpy(to, &v, 16);
                    } else {
#pragma unroll
                        for (int e = 0; e < 4; ++e)
                            if (n + e < columns) to[e] = v[e];
                    }
                }
        }
    } else {
        // 16 x 16: lane group g has columns 4 g .. 4 g + 3 of a row in every block.  Of two blocks side by side, even
        // groups give their part of the second for their odd neighbour's of the first: eight columns of one block each.
        static_assert(FN % 2 == 0 && sizeof(Out) == 2, "pairs of blocks in bf16");
        const int g = lane >> 4;
#pragma unroll
        for (int i = 0; i < FM; ++i) {
            const int m = m0 + 16 * i + (lane & 15);
#pragma unroll
            for (int j = 0; j < FN; j += 2) {
                uint32_t a[2], b[2];
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    a[h] = from_f32<Out>(acc[i][j][2 * h]).bits | (uint32_t)from_f32<Out>(acc[i][j][2 * h + 1]).bits << 16;
                    b[h] = from_f32<Out>(acc[i][j + 1][2 * h]).bits | (uint32_t)from_f32<Out>(acc[i][j + 1][2 * h + 1]).bits << 16;
                    // odd rows of 16 lanes of a <-> even ones of b
                    const auto s = __builtin_amdgcn_permlane16_swap(a[h], b[h], false, false);
                    a[h] = s[0], b[h] = s[1];
                }
                const int n = j0 + 16 * (j + (g & 1)) + 8 * (g >> 1);
                if (m >= rows || n >= columns) continue;
                Out* to = y + m * ld + n;
                if (n + 8 <= columns) {
                    const u32x4 v = {a[0], a[1], b[0], b[1]};
                    __builtin_memcpy(to, &v, 16);
                } else {
#pragma unroll
                    for (int e = 0; e < 8; ++e)
                        if (n + e < columns) to[e] = Out{(uint16_t)((e < 4 ? a[e >> 1 & 1] : b[e >> 1 & 1]) >> (e & 1 ? 16 : 0))};
                }
            }
        }
    }
}

template <int BM, int BN> constexpr int chain_lds() { return (3 * BM + 2 * BN) * 128; }

// Tiles `start`, start + hop, ... of the product.
template <class Mul, bool AACROSS, bool BACROSS, int EPI, int BM, int BN, int WM, int WN>
__device__ __forceinline__ void chain(const LossProductArgs& p, uint8_t* smem, int start, int hop)
{
    static_assert(WM * WN == 8 && BM % (32 * WM) == 0 && BN % (32 * WN) == 0, "eight waves of 32 x 32 blocks");
    constexpr int E = Mul::E, BK = 128 / E, T = Mul::T, FM = BM / WM / T, FN = BN / WN / T;
    constexpr int A_TILE = BM * 128, B_TILE = BN * 128;

    const int mt = (p.M + BM - 1) / BM, nt = (p.N + BN - 1) / BN, total = mt * nt;
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int wm = wave / WN * T * FM, wn = wave % WN * T * FN;
    const int steps = p.K > 0 ? (p.K + BK - 1) / BK : 1;       // without terms one step of zeros

    Stream<E, AACROSS, BM, false> sa;
    Stream<E, BACROSS, BN, false> sb;
    auto start_a = [&](int id) {
        int tm, tn;
        pick_tile(id, mt, nt, tm, tn);
        sa.start(p.a, p.lda, nullptr, 0, tm * BM, AACROSS ? p.a_rows : p.M, 0, AACROSS ? p.K : p.a_K, wave, lane);
    };
    auto start_b = [&](int id) {
        int tm, tn;
        pick_tile(id, mt, nt, tm, tn);
        sb.start(p.b, p.ldb, nullptr, 0, tn * BN, BACROSS ? p.b_rows : p.N, 0, BACROSS ? p.K : p.a_K, wave, lane);
    };
    uint8_t* const b_tiles = smem + 3 * A_TILE;
    // the tile and step of A or B whose loads come next
    int id_a = start, id_b = start, next_a = 0, next_b = 0;
    start_a(id_a);
    start_b(id_b);
    auto turn_a = [&] {
        if (next_a == steps) {
            next_a = 0, id_a += hop;
            if (id_a < total) start_a(id_a);
        }
        sa.next(id_a < total);
        ++next_a;
    };
    auto turn_b = [&] {
        if (next_b == steps) {
            next_b = 0, id_b += hop;
            if (id_b < total) start_b(id_b);
        }
        sb.next(id_b < total);
        ++next_b;
    };

    using Block = typename Mul::Block;
    constexpr int V = T / 16;                                  // vectors of a fragment's half
    u32x4 fa[2][FM][V], fb[2][FN][V];
    Block acc[FM][FN];
    // reads, products and loads of a half step as in linear_fast.h
    constexpr int READS = V * (FM + FN), PRODUCTS = FM * FN;
    auto read = [&](const uint8_t* ta, const uint8_t* tb, int s, int q) {
        const int t = q < V * (FN + 1) ? q / (FN + 1) : q % V;
        const int i = q < V * (FN + 1) ? q % (FN + 1) - FN : q / V - FN;
        if (i < 0) fb[s][i + FN][t] = read_piece<E, BACROSS, T>(tb, wn + T * (i + FN), s, t, lane);
        else fa[s][i][t] = read_piece<E, AACROSS, T>(ta, wm + T * i, s, t, lane);
    };
    auto half = [&](int s, const uint8_t* ta, const uint8_t* tb, auto& stream, uint8_t* into, auto&& turn) {
        constexpr int LOADS = std::remove_reference_t<decltype(stream)>::N;
#pragma unroll
        for (int n = 0; n < PRODUCTS; ++n) {
            const int i = n / FN, j = n % FN;
            acc[i][j] = Mul::block(fb[s][j], fa[s][i], acc[i][j]);
#pragma unroll
            for (int q = 0; q < READS; ++q)
                if (q * PRODUCTS * 3 / (READS * 4) == n) read(ta, tb, s ^ 1, q);
#pragma unroll
            for (int l = 0; l < LOADS; ++l)
                if (l * PRODUCTS / (2 * LOADS) == n) stream.issue(into, wave, l);
            if (n == PRODUCTS * 3 / 4) turn();
            __builtin_amdgcn_sched_barrier(0);
        }
    };

    constexpr int LA = BM / 64, LB = BN / 64;
#pragma unroll
    for (int b = 0; b < 2; ++b) {
        turn_a();
#pragma unroll
        for (int l = 0; l < LA; ++l) sa.issue(smem + b * A_TILE, wave, l);
        turn_b();
#pragma unroll
        for (int l = 0; l < LB; ++l) sb.issue(b_tiles + b * B_TILE, wave, l);
    }
    landed<LA + LB>();
#pragma unroll
    for (int q = 0; q < READS; ++q) read(smem, b_tiles, 0, q);
    int a0 = 0, a1 = A_TILE, a2 = 2 * A_TILE;                  // A of this step and the two after it
    int b0 = 0, b1 = B_TILE;
    turn_a();
    for (int id = start; id < total; id += hop) {
#pragma unroll
        for (int i = 0; i < FM; ++i)
#pragma unroll
            for (int j = 0; j < FN; ++j)
#pragma unroll
                for (int e = 0; e < (int)(sizeof(Block) / 4); ++e) acc[i][j][e] = 0.0f;
        for (int t = 0; t < steps; ++t) {
            half(0, smem + a0, b_tiles + b0, sa, smem + a2, turn_b);
            landed<LA>();
            half(1, smem + a1, b_tiles + b1, sb, b_tiles + b0, turn_a);
            const int a = a0;
            a0 = a1, a1 = a2, a2 = a;
            b0 ^= B_TILE, b1 ^= B_TILE;
        }
        int tm, tn;
        pick_tile(id, mt, nt, tm, tn);
        const int m0 = tm * BM + wm, j0 = tn * BN + wn;
        using Out = typename Mul::Out;
        if constexpr (EPI == EPI_LOSS) {
            loss_wave<E == 4>(p, acc, m0, j0, lane);
        } else {
            if constexpr (EPI == EPI_LOGITS_GRAD) {
                gradient_wave<E == 4>(p, acc, m0, j0, lane);
            } else {
                const float unit = loss_unit<E == 4>(p.loss);
#pragma unroll
                for (int i = 0; i < FM; ++i)
#pragma unroll
                    for (int j = 0; j < FN; ++j)
#pragma unroll
                        for (int e = 0; e < (int)(sizeof(Block) / 4); ++e) acc[i][j][e] *= unit;
            }
            store_wave(static_cast<Out*>(p.y), p.ldy, p.M, EPI == EPI_LOGITS_GRAD ? p.y_columns : p.N, acc, m0, j0, lane);
        }
    }
    landed<0>();
}

template <class Mul, bool AACROSS, bool BACROSS, int EPI, int BM, int BN, int WM, int WN>
__global__ __launch_bounds__(FAST_THREADS, 2) void linear_chain_kernel(const LossProductArgs p)
{
    __shared__ __align__(1024) uint8_t smem[chain_lds<BM, BN>()];
    chain<Mul, AACROSS, BACROSS, EPI, BM, BN, WM, WN>(p, smem, blockIdx.x, gridDim.x);
}

// dx and dw side by side: `first` workgroups on dz W, the others on dz^T x.
template <class Mul, int BM, int BN, int WM, int WN>
__global__ __launch_bounds__(FAST_THREADS, 2) void linear_pair_kernel(const LossProductArgs dx, const LossProductArgs dw, int first)
{
    __shared__ __align__(1024) uint8_t smem[chain_lds<BM, BN>()];
    const int id = blockIdx.x;
    if (id < first) chain<Mul, false, true, EPI_STORE, BM, BN, WM, WN>(dx, smem, id, first);
    else chain<Mul, true, true, EPI_STORE, BM, BN, WM, WN>(dw, smem, id - first, gridDim.x - first);
}

}  // namespace miconv
