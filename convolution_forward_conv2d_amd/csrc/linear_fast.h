// linear_fast.h -- the product with its epilogue on large tiles, for operands
// whose rows are 16-byte aligned multiples of 16 bytes (the host packs others
// first, or takes linear_any.hip).
//
// Eight waves on a tile of BM x BN, one workgroup per CU.  Operands go from
// memory straight into LDS (buffer loads with an LDS destination, 16 bytes a
// lane): A has three buffers there, B two, 160 KB at 256 x 256.  From LDS they
// pass into the matrix instructions' fragments, double-buffered in registers by
// half steps:
//
//   half 0   products of half 0, reading half 1 of step t, loading A of t + 2
//   barrier  A and B of step t + 1 have landed, nobody reads step t's any more
//   half 1   products of half 1, reading half 0 of step t + 1, loading B of t + 2
//
// Reads and loads are placed one by one between the matrix instructions: a CU
// takes a load instruction's kilobyte in about 16 cycles, so loads issued
// together hold up the products behind them (by half of their own time at
// 256 x 256), and over both halves they use at most half of that rate.  A load
// of A has two halves to arrive after its own, one of B one and a half (a half:
// 1024 cycles at 256 x 256).
//
// What bounds it is power: bf16 8192^3 takes 754 us (1458 TFLOP/s) with the
// matrix units busy 70% of the cycles at 1.8 GHz of 2.4, and 605 us on zeros.
// So what moves fewer bits wins: the 16 x 16 x 32 instruction, whose blocks'
// sums pass through the registers half as often for the same work as 32 x 32 x
// 16's, took 846 us to 778.  fp32 (tiles up to 128 x 128, two workgroups a CU)
// is bound by its matrix instructions: 119 TFLOP/s of 157 at 4096^3.
#pragma once

#include <type_traits>

#include "linear_tile.h"
#include "kernels.h"

namespace miconv {

constexpr int FAST_THREADS = 512;

typedef __attribute__((address_space(3))) void* lds_ptr;
typedef int i32x4 __attribute__((ext_vector_type(4)));

// 16 bytes a lane from the descriptor's memory at `offset` into LDS at `to` + 16 * lane; past the descriptor's end:
// zeros.  In assembly because the compiler waits for every load into LDS before each transposing LDS read that follows,
// whatever the two touch (the gradients' products ran at half speed); the kernel's own waits (landed) order them.
// Nothing arrives in a register, and the inputs are read when the instruction issues.  m0 is a register the compiler only
// ever sets itself right before an instruction that takes it, and nothing else here does; the no-op is the state it needs.
__device__ __forceinline__ void load_to_lds(i32x4 rsrc, uint32_t offset, uint32_t to)
{
    asm volatile("s_mov_b32 m0, %2\n\ts_nop 0\n\tbuffer_load_dwordx4 %0, %1, 0 offen lds" ::"v"(offset), "s"(rsrc), "s"(to)
                 : "memory");
}

// One operand's loads: R lines of 128 bytes a step, 8 lines per wave
// instruction, R / 64 instructions per wave (instruction i of wave w: lines
// 8 (w + 8 i) on).  Everything that differs between waves and instructions is
// scalar, one offset per lane serves all of them.  The buffer descriptors end
// where the operand ends, so rows past it (and, stored across, k past K) load
// as zeros.
template <int E, bool ACROSS, int R, bool GATED> struct Stream {
    static constexpr int N = R / 64, LINES = 128 / E;
    const uint8_t* base;         // this wave's first line at the current step's k
    int64_t advance;             // bytes per step
    int64_t left;                // bytes from base to the operand's end
    uint32_t hop;                // bytes between this wave's instructions
    uint32_t off;
    int k_left;                  // reduction elements from the current step on
    int k_lane;                  // this lane's first element of a step (k-major)

    __device__ __forceinline__ void start(const uint8_t* p, int64_t ld, const uint8_t* p2, int64_t ld2, int r0, int rows,
                                          int k0, int K, int wave, int lane)
    {
        k_left = K - k0;
        const int line = wave * 8 + (lane >> 3);               // of instruction 0
        int piece;
        if constexpr (ACROSS) {
            // panel of line: line / LINES; a wave's k within the panel does not depend on the instruction
            const int panel = wave * 8 / LINES, k = k0 + wave * 8 % LINES;
            base = p + (int64_t)r0 * E + panel * 128 + (int64_t)k * ld;
            left = (int64_t)(K - 1 - k) * ld + (int64_t)(rows - r0) * E - panel * 128;
            hop = 64 / LINES * 128;
            advance = ld * LINES;
            piece = E == 2 ? (lane & 7) ^ ((line & 2) << 1) ^ ((line & 8) >> 2) : lane & 7;
        } else {
            int r = r0 + wave * 8;
            hop = 64 * (uint32_t)ld;
            if constexpr (GATED) {
                // raw rows: 16 of the gate's, 16 of the other's; 64 raw rows are 32 of each, so a wave keeps to one
                if (wave & 2) p = p2, ld = ld2;
                r = r0 / 2 + (wave >> 2) * 16 + (wave & 1) * 8;
                hop = 32 * (uint32_t)ld;
            }
            base = p + (int64_t)r * ld + (int64_t)k0 * E;
            left = (int64_t)(rows - 1 - r) * ld + (((int64_t)K * E + 15) & ~15ll) - (int64_t)k0 * E;
            advance = 128;
            piece = (lane & 7) ^ ((line >> 1) & 7);
        }
        k_lane = piece * (16 / E);
        off = (uint32_t)((lane >> 3) * ld + piece * 16);
    }

    // The current step's loads (nothing is fetched unless `some`), then on to the next step.
    i32x4 rsrc;
    uint32_t at;
    __device__ __forceinline__ void next(bool some)
    {
        const int records = (int)(left < 0 || !some ? 0 : left > 0x7fffff00 ? 0x7fffff00 : left);
        const uint64_t from = reinterpret_cast<uint64_t>(base);
        rsrc = i32x4{(int)from, (int)(from >> 32) & 0xffff, records, 0x00020000};
        asm volatile("s_nop 4" : "+s"(rsrc));                  // the states a vector-written scalar would need before a load
        at = off;
        // a row's end is not the operand's: pieces past K take an offset no descriptor reaches (the host keeps pitches
        // below 4 MB, so offsets within a tile stay below 2^30 and the sum does not wrap)
        if constexpr (!ACROSS) at = k_lane < k_left ? off : 0x80000000u;
        base += advance;
        left -= advance;
        k_left -= LINES;
    }
    __device__ __forceinline__ void issue(uint8_t* tile, int wave, int i) const
    {
        load_to_lds(rsrc, at + i * hop, (uint32_t)(uintptr_t)(lds_ptr)(tile + wave * 1024 + i * 8192));
    }
};

// All but this wave's last PENDING loads have landed in LDS and its reads are done, then everyone's.
template <int PENDING> __device__ __forceinline__ void landed()
{
    static_assert(PENDING < 16, "the low four bits of vmcnt");
    __builtin_amdgcn_sched_barrier(0);
    asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)\n\ts_barrier" ::"n"(PENDING) : "memory");
    __builtin_amdgcn_sched_barrier(0);
}

template <class Mul, bool AACROSS, bool BACROSS, int EPI, int BM, int BN, int WM, int WN>
__global__ __launch_bounds__(FAST_THREADS, 2) void linear_fast_kernel(const ProductArgs p)
{
    static_assert(WM * WN == 8 && BM % (32 * WM) == 0 && BN % (32 * WN) == 0, "eight waves of 32 x 32 blocks");
    constexpr int E = Mul::E, BK = 128 / E, T = Mul::T, FM = BM / WM / T, FN = BN / WN / T;
    constexpr int A_TILE = BM * 128, B_TILE = BN * 128, LDS = 3 * A_TILE + 2 * B_TILE;
    constexpr bool GATED = EPI == EPI_GATED;
    static_assert(8 * 32 * (T * FN + 4) * 4 <= LDS, "the epilogue's stages fit");
    __shared__ __align__(1024) uint8_t smem[LDS];

    const int raw_n = GATED ? gated_raw_columns(p.N) : p.N;
    const int mt = (p.M + BM - 1) / BM, nt = (raw_n + BN - 1) / BN;
    int tm, tn;
    pick_tile(blockIdx.x, mt, nt, tm, tn);
    const int m0 = tm * BM, j0 = tn * BN;
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int wm = wave / WN * T * FM, wn = wave % WN * T * FN;

    const int per_segment = (p.K + BK - 1) / BK;
    const int steps = per_segment * p.k_segments;
    const int first = (int)((int64_t)steps * blockIdx.z / p.splits);
    const int last = (int)((int64_t)steps * (blockIdx.z + 1) / p.splits);

    constexpr bool SEGMENTS = EPI == EPI_PLAIN && !AACROSS && BACROSS;   // dx of a gated layer: two of k
    Stream<E, AACROSS, BM, false> sa, sa2;
    Stream<E, BACROSS, BN, GATED> sb, sb2;
    const int seg = first >= per_segment;
    const int k0 = (first - seg * per_segment) * BK;
    sa.start(p.a + (int64_t)seg * p.k_pitch * E, p.lda, nullptr, 0, m0, AACROSS ? p.a_rows : p.M, k0,
             AACROSS ? p.K : p.a_K, wave, lane);
    sb.start(seg ? p.b2 : p.b, p.ldb, p.b2, p.ldb2, j0, BACROSS ? p.b_rows : p.N, k0,
             BACROSS ? p.K : p.a_K, wave, lane);
    if constexpr (SEGMENTS) {
        sa2.start(p.a + (int64_t)p.k_pitch * E, p.lda, nullptr, 0, m0, p.M, 0, p.a_K, wave, lane);
        sb2.start(p.b2, p.ldb, nullptr, 0, j0, p.b_rows, 0, p.K, wave, lane);
    }
    uint8_t* const b_tiles = smem + 3 * A_TILE;
    // the loads of the next step of A or B not loaded yet
    int next_a = first, next_b = first;
    auto turn_a = [&] {
        if constexpr (SEGMENTS) {
            const bool turn = next_a == per_segment;           // selects, no branch: the pitches are the same
            sa.base = turn ? sa2.base : sa.base, sa.left = turn ? sa2.left : sa.left;
            sa.k_left = turn ? sa2.k_left : sa.k_left;
        }
        sa.next(next_a < last);
        ++next_a;
    };
    auto turn_b = [&] {
        if constexpr (SEGMENTS) {
            const bool turn = next_b == per_segment;
            sb.base = turn ? sb2.base : sb.base, sb.left = turn ? sb2.left : sb.left;
        }
        sb.next(next_b < last);
        ++next_b;
    };

    using Block = typename Mul::Block;
    Block acc[FM][FN];
#pragma unroll
    for (int i = 0; i < FM; ++i)
#pragma unroll
        for (int j = 0; j < FN; ++j)
#pragma unroll
            for (int e = 0; e < (int)(sizeof(Block) / 4); ++e) acc[i][j][e] = 0.0f;

    constexpr int V = T / 16;                                  // vectors of a fragment's half
    u32x4 fa[2][FM][V], fb[2][FN][V];
    // read q of the fragments of half s, in the order the products need them
    constexpr int READS = V * (FM + FN);
    auto read = [&](const uint8_t* ta, const uint8_t* tb, int s, int q) {
        const int t = q < V * (FN + 1) ? q / (FN + 1) : q % V;
        const int i = q < V * (FN + 1) ? q % (FN + 1) - FN : q / V - FN;             // A's block, or < 0: B's i + FN
        if (i < 0) fb[s][i + FN][t] = read_piece<E, BACROSS, T>(tb, wn + T * (i + FN), s, t, lane);
        else fa[s][i][t] = read_piece<E, AACROSS, T>(ta, wm + T * i, s, t, lane);
    };
    // One half step: its products, with the next half's reads and one operand's loads between them, and late in it the
    // other operand's descriptor for the half after: in front of that half's products it held up both waves of a SIMD.
    constexpr int PRODUCTS = FM * FN;
    auto half = [&](int s, const uint8_t* ta, const uint8_t* tb, auto& stream, uint8_t* into, auto&& turn) {
        constexpr int LOADS = std::remove_reference_t<decltype(stream)>::N;
#pragma unroll
        for (int n = 0; n < PRODUCTS; ++n) {
            const int i = n / FN, j = n % FN;
            acc[i][j] = Mul::block(fb[s][j], fa[s][i], acc[i][j]);
            // reads in the first three quarters of the slots, so the barrier does not wait for them
#pragma unroll
            for (int q = 0; q < READS; ++q)
                if (q * PRODUCTS * 3 / (READS * 4) == n) read(ta, tb, s ^ 1, q);
            // loads in the first half of the slots
#pragma unroll
            for (int l = 0; l < LOADS; ++l)
                if (l * PRODUCTS / (2 * LOADS) == n) stream.issue(into, wave, l);
            if (n == PRODUCTS * 3 / 4) turn();
            __builtin_amdgcn_sched_barrier(0);
        }
    };

    if (first < last) {
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
        int a0 = 0, a1 = A_TILE, a2 = 2 * A_TILE;              // A of steps t, t + 1, t + 2
        int b0 = 0, b1 = B_TILE;
        turn_a();
        for (int t = first; t < last; ++t) {
            half(0, smem + a0, b_tiles + b0, sa, smem + a2, turn_b);
            landed<LA>();
            half(1, smem + a1, b_tiles + b1, sb, b_tiles + b0, turn_a);
            const int a = a0;
            a0 = a1, a1 = a2, a2 = a;
            b0 ^= B_TILE, b1 ^= B_TILE;
        }
        landed<0>();
    }
    finish_wave<typename Mul::Out, EPI>(p, reinterpret_cast<float*>(smem) + wave * 32 * (T * FN + 4), acc,
                                                m0 + wm, j0 + wn, blockIdx.z, lane);
}

}  // namespace miconv
