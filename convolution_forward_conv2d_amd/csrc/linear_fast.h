// linear_fast.h -- the product with its epilogue on large tiles, for operands
// whose rows are 16-byte aligned multiples of 16 bytes (the host packs others
// first, or takes linear_any.hip).
//
// Eight waves on a tile of BM x BN, one workgroup per CU.  Operands go from
// memory straight into LDS (buffer loads with an LDS destination, 16 bytes a
// lane), double-buffered, and from there into the matrix instructions'
// fragments, which are double-buffered in registers by half steps:
//
//   half 0   read fragments of half 1 of step t       products of half 0
//   barrier  step t + 1 has landed, nobody reads step t's buffer any more
//   half 1   start loading step t + 2, read half 0 of step t + 1
//                                                     products of half 1
//
// so the products wait for neither memory nor LDS, and a load has a whole step
// (2048 cycles at 256 x 256) to arrive.
#pragma once

#include "linear_tile.h"
#include "kernels.h"

namespace miconv {

constexpr int FAST_THREADS = 512;

typedef __attribute__((address_space(3))) void* lds_ptr;

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
            piece = E == 2 ? (lane & 7) ^ ((line & 2) << 1) : lane & 7;
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

    // Loads of the current step into `tile` (nothing is fetched unless `some`), then on to the next step.
    __device__ __forceinline__ void load(uint8_t* tile, int wave, bool some)
    {
        // the host keeps pitches below 4 MB: offsets within a tile stay below 2^30
        const int records = (int)(left < 0 || !some ? 0 : left > 0x7fffff00 ? 0x7fffff00 : left);
        const uint8_t* at = base;
        uint32_t o = off;
        if constexpr (!ACROSS) {
            // a row's end is not the operand's: pieces past K take an offset no descriptor reaches
            o = k_lane < k_left ? o : 0xfffffff0u;
        }
#pragma unroll
        for (int i = 0; i < N; ++i) {
            const int here = records - (int)(i * hop);
            auto rs = __builtin_amdgcn_make_buffer_rsrc(const_cast<uint8_t*>(at), 0, here > 0 ? here : 0, 0x00020000);
            __builtin_amdgcn_raw_ptr_buffer_load_lds(rs, (lds_ptr)(tile + wave * 1024 + i * 8192), 16, o, 0, 0, 0);
            at += hop;
        }
        base += advance;
        left -= advance;
        k_left -= LINES;
    }
};

// This wave's loads into LDS have landed, then everyone's.
__device__ __forceinline__ void landed()
{
    __builtin_amdgcn_s_waitcnt(0x0f70);                        // vmcnt(0)
    __syncthreads();
}

template <class Mul, bool AACROSS, bool BACROSS, int EPI, int BM, int BN, int WM, int WN>
__global__ __launch_bounds__(FAST_THREADS, 2) void linear_fast_kernel(const ProductArgs p)
{
    static_assert(WM * WN == 8 && BM % (32 * WM) == 0 && BN % (32 * WN) == 0, "eight waves of 32 x 32 blocks");
    constexpr int E = Mul::E, BK = 128 / E, FM = BM / WM / 32, FN = BN / WN / 32;
    constexpr int STEP = (BM + BN) * 128;
    constexpr bool GATED = EPI == EPI_GATED;
    static_assert(8 * 32 * (32 * FN + 4) * 4 <= 2 * STEP, "the epilogue's stages fit");
    __shared__ __align__(1024) uint8_t smem[2 * STEP];

    const int raw_n = GATED ? gated_raw_columns(p.N) : p.N;
    const int mt = (p.M + BM - 1) / BM, nt = (raw_n + BN - 1) / BN;
    int tm, tn;
    pick_tile(blockIdx.x, mt, nt, tm, tn);
    const int m0 = tm * BM, j0 = tn * BN;
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int wm = wave / WN * 32 * FM, wn = wave % WN * 32 * FN;

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
    int next = first;
    auto load = [&](int buf) {                                 // the next step not loaded yet
        if constexpr (SEGMENTS) {
            const bool turn = next == per_segment;             // selects, no branch: the pitches are the same
            sa.base = turn ? sa2.base : sa.base, sa.left = turn ? sa2.left : sa.left;
            sb.base = turn ? sb2.base : sb.base, sb.left = turn ? sb2.left : sb.left;
            sa.k_left = turn ? sa2.k_left : sa.k_left;
        }
        sa.load(smem + buf * BM * 128, wave, next < last);
        sb.load(smem + (2 * BM + buf * BN) * 128, wave, next < last);
        ++next;
    };

    f32x16 acc[FM][FN];
#pragma unroll
    for (int i = 0; i < FM; ++i)
#pragma unroll
        for (int j = 0; j < FN; ++j)
#pragma unroll
            for (int e = 0; e < 16; ++e) acc[i][j][e] = 0.0f;

    u32x4 fa[2][FM][2], fb[2][FN][2];
    auto read = [&](int buf, int s) {
        // A's two buffers, then B's: either is within an LDS instruction's offset of one address
        const uint8_t* ta = smem + buf * BM * 128;
        const uint8_t* tb = smem + (2 * BM + buf * BN) * 128;
#pragma unroll
        for (int j = 0; j < FN; ++j) read_fragment<E, BACROSS>(tb, wn + 32 * j, s, lane, fb[s][j]);
#pragma unroll
        for (int i = 0; i < FM; ++i) read_fragment<E, AACROSS>(ta, wm + 32 * i, s, lane, fa[s][i]);
    };
    auto multiply = [&](int s) {
#pragma unroll
        for (int i = 0; i < FM; ++i)
#pragma unroll
            for (int j = 0; j < FN; ++j) acc[i][j] = Mul::mfma(fb[s][j], fa[s][i], acc[i][j]);
    };

    // One LDS read (two where rows are read across) before each of the first products: the reads are spread over the
    // half step in which they have to arrive, and so are the loads.
    constexpr int PRODUCTS = FM * FN * Mul::PER_HALF, LOADS = (BM + BN) / 64;
    constexpr int READS = FM * (AACROSS ? 2 * E : 2) + FN * (BACROSS ? 2 * E : 2);
    auto pace = [&](bool loads) {
#pragma unroll
        for (int i = 0; i < PRODUCTS; ++i) {
            __builtin_amdgcn_sched_group_barrier(0x100, (READS + PRODUCTS - 1) / PRODUCTS, 0);
            if (loads && i < LOADS) __builtin_amdgcn_sched_group_barrier(0x020, 1, 0);
            __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);
        }
    };

    if (first < last) {
        load(0);
        landed();
        load(1);
        read(0, 0);
        auto step = [&](int buf) {
            read(buf, 1);
            multiply(0);
            pace(false);
            __builtin_amdgcn_sched_barrier(0);
            landed();
            __builtin_amdgcn_sched_barrier(0);
            read(buf ^ 1, 0);
            load(buf);                                         // past the last step: nothing
            multiply(1);
            pace(true);
            __builtin_amdgcn_sched_barrier(0);
        };
        int t = first;
        for (; t + 1 < last; t += 2) {
            step(0);
            step(1);
        }
        if (t < last) step(0);
        landed();
    }
    finish_wave<typename Mul::Out, EPI, FM, FN>(p, reinterpret_cast<float*>(smem) + wave * 32 * (32 * FN + 4), acc,
                                                m0 + wm, j0 + wn, blockIdx.z, lane);
}

}  // namespace miconv
