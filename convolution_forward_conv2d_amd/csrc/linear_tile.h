// linear_tile.h -- one workgroup's tile of a product in LDS: its layouts, the
// fragments the matrix instructions take from it, and the epilogue.
//
// A k step of a tile is 128 bytes of each of its rows, R x 128 bytes in LDS:
//  * k-major operand: row r's 128 bytes together, its 16-byte pieces permuted
//    by (r / 2) % 8, so that sixteen rows read at one k meet all 64 banks;
//  * operand stored across k: panels of 128 bytes of rows (64 bf16, 32 fp32),
//    each with one 128-byte line per k.  bf16 is read with the LDS's
//    transposing loads, four lines of 64 bytes or eight (four and four, eight
//    apart) of 32 at a time: the two 64-byte halves of a line swap places where
//    k & 2 is set and their 32-byte halves where k & 8 is, so either meets all
//    64 banks.
// Either way eight lines of 128 bytes are 1 KB, one load instruction's worth.
#pragma once

#include "linear_common.h"

namespace miconv {

// byte offset in the tile of the 16-byte piece `piece` of line `line` (k-major:
// line = row; across k: line = panel * lines per panel + k)
template <int E, bool ACROSS> __device__ __forceinline__ int tile_piece(int line, int piece)
{
    if constexpr (!ACROSS) return line * 128 + 16 * (piece ^ ((line >> 1) & 7));
    if constexpr (E == 2) return line * 128 + 16 * (piece ^ ((line & 2) << 1) ^ ((line & 8) >> 2));
    return line * 128 + 16 * piece;
}

// Fragment of T rows from r0 (a multiple of T), half `s` of the step: its vector t of T / 16.
template <int E, bool ACROSS, int T>
__device__ __forceinline__ u32x4 read_piece(const uint8_t* tile, int r0, int s, int t, int lane)
{
    constexpr int G = 64 / T;                                  // lane groups, each at another 16 bytes of k
    const int group = lane / T;
    if constexpr (!ACROSS) {
        const int r = r0 + lane % T;
        return *reinterpret_cast<const u32x4*>(tile + tile_piece<E, false>(r, 4 * s + G * t + group));
    } else if constexpr (E == 2) {
        // sixteen lanes fetch 4 k x 16 rows, 8 bytes each, and get one row's four k
        typedef short s16x4 __attribute__((ext_vector_type(4)));
        typedef __attribute__((address_space(3))) s16x4* lds4;
        const int j = lane & 15;
        const int k = 8 * group + (j >> 2);
        const int byte = ((r0 & 48) << 1) + (T == 32 ? (lane & 16) << 1 : 0) + 8 * (j & 3);
        const uint8_t* at = tile + (r0 >> 6) * 8192 + (32 * s + 16 * t + k) * 128 + (byte ^ ((k & 2) << 5) ^ ((k & 8) << 2));
        const u32x2 lo = __builtin_bit_cast(u32x2, __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds4)at));
        const u32x2 hi = __builtin_bit_cast(u32x2, __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds4)(at + 512)));
        return u32x4{lo[0], lo[1], hi[0], hi[1]};
    } else {
        static_assert(T == 32, "fp32 blocks");
        const uint8_t* at = tile + (r0 >> 5) * 4096 + (16 * s + 8 * t + 4 * group) * 128 + 4 * (lane & 31);
        u32x4 f;
#pragma unroll
        for (int e = 0; e < 4; ++e) f[e] = *reinterpret_cast<const uint32_t*>(at + e * 128);
        return f;
    }
}

template <int E, bool ACROSS>
__device__ __forceinline__ void read_fragment(const uint8_t* tile, int r0, int s, int lane, u32x4 (&f)[2])
{
#pragma unroll
    for (int t = 0; t < 2; ++t) f[t] = read_piece<E, ACROSS, 32>(tile, r0, s, t, lane);
}

// Lanes exchange data through LDS next: the wave's DS instructions execute in
// order, this keeps the compiler from moving them across.
__device__ __forceinline__ void wave_order()
{
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    __builtin_amdgcn_wave_barrier();
}

// The epilogue of 32 rows of W raw columns, all of which exist, from the wave's
// stage.  A lane keeps its eight columns from pass to pass (with 96 columns four
// lanes stay idle), so bias and column scales are loaded once per tile; a row's
// scale comes from the lane that loaded it.  A residual is added in a pass of
// its own, unrolled, so that its loads are in flight together: one load after
// the other, as in the general form, costs a tile of 256 x 256 about 13 us (526
// us instead of 500 on 8192 x 4096 x 9216 with a residual).
template <class Out, int EPI, int W> struct WholeRows {
    static constexpr bool GATED = EPI == EPI_GATED, EXACT = sizeof(Out) == 4;
    static constexpr int PER = GATED ? W / 16 : W / 8, ROWS = 64 / PER, PASSES = (32 + ROWS - 1) / ROWS, PITCH = W + 4;
    static constexpr int PIECES = sizeof(Out) / 2;             // of 16 bytes, in eight values
    struct Columns {
        float bias[8], scale[8], scale2[8];
    };
    int row, n;                  // of the first pass
    int at;                      // column in the stage
    __device__ __forceinline__ WholeRows(int lane, int n0)
    {
        row = lane < ROWS * PER ? lane / PER : 32;             // past the last row: idle
        const int g = lane % PER;
        n = n0 + 8 * g;
        at = GATED ? (g >> 1) * 32 + (g & 1) * 8 : 8 * g;      // group g: block g / 2, its half g % 2
    }
    __device__ __forceinline__ Columns columns(const ProductArgs& p) const
    {
        Columns c;
        if (p.bias) load8(static_cast<const Out*>(p.bias) + n, 8, c.bias);
        if (p.w_scale) load8(p.w_scale + n, 8, c.scale);
        if (GATED && p.w2_scale) load8(p.w2_scale + n, 8, c.scale2);
        return c;
    }
    // Whether all scales of the tile are within 2^-62 and 2^63, so that any two multiply to a normal number.  finish()
    // takes those products as they are; other tiles go the general way, whose scaled() is twice the work (in finish() it
    // was 1.5 percent of 4096 x 9216 x 4096, and a branch there, for its instructions' fetch alone, 1).
    template <int N> __device__ static __forceinline__ bool moderate(const Columns& c, const float (&row_scale)[N])
    {
        bool far = false;
        auto look = [&](float s) { far |= (__float_as_uint(s) << 1) - (65u << 24) >= (125u << 24); };
#pragma unroll
        for (int i = 0; i < N; ++i) look(row_scale[i]);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            look(c.scale[i]);
            if constexpr (GATED) look(c.scale2[i]);
        }
        return __builtin_amdgcn_ballot_w64(far) == 0;
    }
    __device__ __forceinline__ void load(const ProductArgs& p, u32x4 (&res)[PASSES][PIECES], int m0) const
    {
#pragma unroll
        for (int k = 0; k < PASSES; ++k) {
            const int m = min(m0 + min(row + k * ROWS, 31), p.M - 1);
            __builtin_memcpy(res[k], static_cast<const Out*>(p.residual) + (int64_t)m * p.ldr + n, 16 * PIECES);
        }
    }
    __device__ __forceinline__ void finish(const ProductArgs& p, float* stage, const Columns& c,
                                           const u32x4 (&res)[PASSES][PIECES], int m0, float row_scale) const
    {
        const bool adds = p.residual != nullptr;
        const int rows = min(32, p.M - m0);
        if (!adds || p.act != ACT_NONE || p.x_scale || p.bias || p.pre) {
#pragma unroll 1
            for (int r = row; r - row < PASSES * ROWS; r += ROWS) {
                const float xs = __shfl(row_scale, r & 31);
                if (r >= rows) continue;
                float* s = stage + r * PITCH + at;
                float v[8], u[8];
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    v[e] = s[e];
                    if constexpr (GATED) u[e] = s[16 + e];
                }
                if (p.x_scale) {
#pragma unroll
                    for (int e = 0; e < 8; ++e) {
                        v[e] *= xs * c.scale[e];
                        if constexpr (GATED) u[e] *= xs * c.scale2[e];
                    }
                }
                if (!GATED && p.bias) {
#pragma unroll
                    for (int e = 0; e < 8; ++e) v[e] += c.bias[e];
                }
                if (p.pre) store8(static_cast<Out*>(p.pre) + (int64_t)(m0 + r) * p.ldp + n, 8, v);
                if (GATED && p.pre2) store8(static_cast<Out*>(p.pre2) + (int64_t)(m0 + r) * p.ldp2 + n, 8, u);
                activate8<EXACT>(p.act, v);
                if constexpr (GATED) {
#pragma unroll
                    for (int e = 0; e < 8; ++e) v[e] *= u[e];
                }
                if (adds) {
#pragma unroll
                    for (int e = 0; e < 8; ++e) s[e] = v[e];
                } else {
                    store8(static_cast<Out*>(p.y) + (int64_t)(m0 + r) * p.ldy + n, 8, v);
                }
            }
        }
        if (adds) {
            wave_order();
#pragma unroll
            for (int k = 0; k < PASSES; ++k) {
                const int r = row + k * ROWS;
                if (r >= rows) continue;
                const float* s = stage + r * PITCH + at;
                Out x[8];
                __builtin_memcpy(x, res[k], sizeof(x));
                float v[8];
#pragma unroll
                for (int e = 0; e < 8; ++e) v[e] = s[e] + to_f32(x[e]);
                store8(static_cast<Out*>(p.y) + (int64_t)(m0 + r) * p.ldy + n, 8, v);
            }
        }
    }
};

// Epilogue of one wave: its FM x FN blocks of T rows x T raw columns (T = 16 or
// 32), first row m0, first raw column j0.  acc holds columns along its registers, so a
// lane writes four columns of a row at once into the wave's own LDS stage and
// then takes eight of a row from it: 16-byte accesses to every tensor, whole
// 64- or 128-byte lines per row.  The caller has passed a barrier after the
// last read of the operand tiles.
template <class Out, int EPI, class Block, int FM, int FN>
__device__ __forceinline__ void finish_wave(const ProductArgs& p, float* stage, Block (&acc)[FM][FN], int m0, int j0,
                                            int split, int lane)
{
    constexpr int T = sizeof(Block) == sizeof(f32x16) ? 32 : 16, W = T * FN, PITCH = W + 4, ROWS = T * FM;
    static_assert(ROWS % 32 == 0, "32 rows at a time");
    // a linear or gated layer's whole tile takes its bias and scales once, and its residual 32 rows ahead
    using Rows = WholeRows<Out, EPI, W>;
    bool whole = EPI != EPI_PLAIN && p.splits == 1 && (EPI == EPI_GATED ? (j0 + W) / 2 : j0 + W) <= p.N;
    const Rows rows(lane, EPI == EPI_GATED ? j0 / 2 : j0);
    typename Rows::Columns columns;
    u32x4 residual[2][Rows::PASSES][sizeof(Out) / 2];
    float row_scale[ROWS / 32];
    if (whole) {
        columns = rows.columns(p);
        if (p.residual) rows.load(p, residual[0], m0);
#pragma unroll
        for (int i = 0; i < ROWS / 32; ++i)
            row_scale[i] = p.x_scale ? p.x_scale[min(m0 + 32 * i + (lane & 31), p.M - 1)] : 1.0f;
    }
#pragma unroll
    for (int i = 0; i < ROWS / 32; ++i) {
#pragma unroll
        for (int j = 0; j < FN; ++j) {
            if constexpr (T == 32) {
#pragma unroll
                for (int q = 0; q < 4; ++q)
                    *reinterpret_cast<f32x4*>(stage + (lane & 31) * PITCH + 32 * j + 8 * q + 4 * (lane >> 5)) =
                        f32x4{acc[i][j][4 * q], acc[i][j][4 * q + 1], acc[i][j][4 * q + 2], acc[i][j][4 * q + 3]};
            } else {
#pragma unroll
                for (int h = 0; h < 2; ++h)
                    *reinterpret_cast<f32x4*>(stage + (16 * h + (lane & 15)) * PITCH + 16 * j + 4 * (lane >> 4)) =
                        acc[2 * i + h][j];
            }
        }
        wave_order();
        // here, where the first rows are in the stage: behind the scales' loads it would wait for them
        if (i == 0 && whole && p.x_scale) whole = Rows::moderate(columns, row_scale);
        if (whole) {
            if (p.residual && i + 1 < ROWS / 32) rows.load(p, residual[(i + 1) & 1], m0 + 32 * i + 32);
            rows.finish(p, stage, columns, residual[i & 1], m0 + 32 * i, row_scale[i]);
        } else if (p.splits > 1) {
            constexpr int PER = W / 8;
#pragma unroll 2
            for (int it = lane; it < 32 * PER; it += 64) {
                const int r = it / PER, c = it % PER * 8, m = m0 + 32 * i + r;
                if (m >= p.M) continue;
                float* out = p.part + ((int64_t)split * p.M + m) * p.part_ld + j0 + c;
#pragma unroll
                for (int h = 0; h < 2; ++h)
                    reinterpret_cast<f32x4*>(out)[h] = reinterpret_cast<const f32x4*>(stage + r * PITCH + c)[h];
            }
        } else if constexpr (EPI == EPI_GATED) {
            constexpr int PER = W / 16;                       // 16 of 32 raw columns are the gate's
#pragma unroll 1
            for (int it = lane; it < 32 * PER; it += 64) {
                const int r = it / PER, g = it % PER;         // group g: block g / 2, its half g % 2
                const float* at = stage + r * PITCH + (g >> 1) * 32 + (g & 1) * 8;
                float v[8], u[8];
#pragma unroll
                for (int e = 0; e < 8; ++e) v[e] = at[e], u[e] = at[16 + e];
                finish8<Out, EPI>(p, m0 + 32 * i + r, j0 / 2 + g * 8, v, u);
            }
        } else {
            constexpr int PER = W / 8;
#pragma unroll 1
            for (int it = lane; it < 32 * PER; it += 64) {
                const int r = it / PER, c = it % PER * 8;
                float v[8], u[8];
#pragma unroll
                for (int e = 0; e < 8; ++e) v[e] = stage[r * PITCH + c + e];
                finish8<Out, EPI>(p, m0 + 32 * i + r, j0 + c, v, u);
            }
        }
        wave_order();
    }
}

// Which tile a workgroup takes.  Workgroups go round the eight XCDs in launch
// order, each with its own L2: an XCD gets a contiguous run of tiles, and the
// run walks GROUP row tiles down before it moves to the next column tile, so
// the 32 tiles an XCD computes at one time share operand rows in its L2.
__device__ __forceinline__ void pick_tile(int id, int mt, int nt, int& tm, int& tn)
{
    constexpr int XCDS = 8, GROUP = 8;
    const int total = mt * nt, per = total / XCDS, rest = total % XCDS;
    const int x = id % XCDS, y = id / XCDS;
    const int t = x * per + (x < rest ? x : rest) + y;
    const int band = t / (GROUP * nt), first = band * GROUP;
    const int rows = mt - first < GROUP ? mt - first : GROUP;
    const int in = t - first * nt;
    tm = first + in % rows;
    tn = in / rows;
}

}  // namespace miconv
