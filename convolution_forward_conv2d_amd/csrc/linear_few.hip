// linear_few.hip -- linear and gated layers on few rows (the next tokens of a
// handful of sequences), any pitches and alignments.
//
// Bound by reading the weights once.  Both kernels keep a weight row's whole
// reduction in one workgroup, so there are no partial sums in memory and no
// second launch, and take weights from memory straight into registers, the next
// turn's loads in flight during this one's products; x comes from L2 the same
// way, rows past M and columns past N repeat the last one and are dropped at
// the end.
//
//  * one or two rows: a wave walks two weight rows (a gated layer: the same row
//    of both products), a kilobyte of each at a time, with fp32 products on the
//    vector units.  One row of 4096 x 9216 bf16 takes 15.1 us, 5.0 TB/s, the
//    rate of a large copy; 9216 x 4096 gated 28.1 us.
//  * up to 32 rows: blocks of 16 rows x 16 columns on the matrix instructions,
//    eight waves taking turns along k, 256 bytes of each weight row, added up
//    in LDS.  Four rows of 4096 x 9216 take 15.3 us (with the first kernel,
//    whose vector work grows with the rows, 20.2; on split tiles 25), sixteen
//    19.5 (25), where reading x again for every 16 columns begins to show.
//
// A cross entropy's logits end here in their rows' statistics, eight columns a
// run: one row of 65536 x 4096 takes 84 us (and 5 to join), eight rows 109.
#include "linear_common.h"
#include "kernels.h"

namespace miconv {

namespace {

constexpr int WAVES = 8;

template <int E> struct Unpack;
template <> struct Unpack<4> {
    static constexpr int N = 4;
    __device__ static void to(u32x4 t, float (&v)[N])
    {
#pragma unroll
        for (int i = 0; i < 4; ++i) v[i] = __uint_as_float(t[i]);
    }
};
template <> struct Unpack<2> {
    static constexpr int N = 8;
    __device__ static void to(u32x4 t, float (&v)[N])
    {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            v[2 * i] = __uint_as_float(t[i] << 16);
            v[2 * i + 1] = __uint_as_float(t[i] & 0xffff0000u);
        }
    }
};
template <> struct Unpack<1> {
    static constexpr int N = 16;
    __device__ static void to(u32x4 t, float (&v)[N])
    {
        typedef float f32x2 __attribute__((ext_vector_type(2)));
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const f32x2 lo = __builtin_amdgcn_cvt_pk_f32_fp8(t[i], false), hi = __builtin_amdgcn_cvt_pk_f32_fp8(t[i], true);
            v[4 * i] = lo[0], v[4 * i + 1] = lo[1], v[4 * i + 2] = hi[0], v[4 * i + 3] = hi[1];
        }
    }
};

template <int E, class Out, int EPI, int MB>
__global__ __launch_bounds__(64 * WAVES) void linear_few_kernel(const ArgsOf<EPI> p)
{
    constexpr bool GATED = EPI == EPI_GATED;
    constexpr int CHUNK = 1024, U = 2;                         // bytes of a row per load, loads of it per turn
    constexpr int COLS = GATED ? WAVES : 2 * WAVES;            // output columns of a workgroup
    __shared__ __align__(16) float sums[2][MB][2 * WAVES];
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int n0 = blockIdx.x * COLS;
    const uint8_t* w[2];
    const uint8_t* x[MB];
    if constexpr (GATED) {
        const int64_t n = min(n0 + wave, p.N - 1);
        w[0] = p.b + n * p.ldb, w[1] = p.b2 + n * p.ldb2;
    } else {
#pragma unroll
        for (int j = 0; j < 2; ++j) w[j] = p.b + (int64_t)min(n0 + 2 * wave + j, p.N - 1) * p.ldb;
    }
#pragma unroll
    for (int i = 0; i < MB; ++i) x[i] = p.a + (int64_t)min(i, p.M - 1) * p.lda;

    float acc[2][MB];
#pragma unroll
    for (int j = 0; j < 2; ++j)
#pragma unroll
        for (int i = 0; i < MB; ++i) acc[j][i] = 0.0f;

    u32x4 fw[2][2][U], fx[2][MB][U];
    auto load = [&](int s, int64_t at) {
#pragma unroll
        for (int u = 0; u < U; ++u) {
#pragma unroll
            for (int j = 0; j < 2; ++j) __builtin_memcpy(&fw[s][j][u], w[j] + at + u * CHUNK + 16 * lane, 16);
#pragma unroll
            for (int i = 0; i < MB; ++i) __builtin_memcpy(&fx[s][i][u], x[i] + at + u * CHUNK + 16 * lane, 16);
        }
    };
    auto multiply = [&](int s) {
        constexpr int V = Unpack<E>::N;
#pragma unroll
        for (int u = 0; u < U; ++u) {
            float a[2][V];
#pragma unroll
            for (int j = 0; j < 2; ++j) Unpack<E>::to(fw[s][j][u], a[j]);
#pragma unroll
            for (int i = 0; i < MB; ++i) {
                float b[V];
                Unpack<E>::to(fx[s][i][u], b);
#pragma unroll
                for (int e = 0; e < V; ++e)
#pragma unroll
                    for (int j = 0; j < 2; ++j) acc[j][i] = fmaf(a[j][e], b[e], acc[j][i]);
            }
        }
    };
    constexpr int TURN = U * CHUNK;
    const int64_t row = (int64_t)p.K * E, whole = row / TURN * TURN;
    int64_t at = 0;
    if (at < whole) load(0, at);
    while (at < whole) {
        if (at + TURN < whole) load(1, at + TURN);
        multiply(0);
        at += TURN;
        if (at >= whole) break;
        if (at + TURN < whole) load(0, at + TURN);
        multiply(1);
        at += TURN;
    }
    if (whole < row) {
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int64_t here = whole + u * CHUNK + 16 * lane;
            const int left = (int)((row - here) / E);
#pragma unroll
            for (int j = 0; j < 2; ++j) fw[0][j][u] = load_piece<E>(w[j] + here, left);
#pragma unroll
            for (int i = 0; i < MB; ++i) fx[0][i][u] = load_piece<E>(x[i] + here, left);
        }
        multiply(0);
    }

#pragma unroll
    for (int j = 0; j < 2; ++j)
#pragma unroll
        for (int i = 0; i < MB; ++i) {
#pragma unroll
            for (int o = 32; o > 0; o >>= 1) acc[j][i] += __shfl_xor(acc[j][i], o);
            if (lane == 0) sums[GATED ? j : 0][i][GATED ? wave : 2 * wave + j] = acc[j][i];
        }
    __syncthreads();
    constexpr int GROUPS = COLS / 8;
    if (threadIdx.x >= MB * GROUPS) return;
    const int m = threadIdx.x / GROUPS, g = threadIdx.x % GROUPS;
    float v[8], u[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) {
        v[e] = sums[0][m][8 * g + e];
        if constexpr (GATED) u[e] = sums[1][m][8 * g + e];
    }
    finish8<Out, EPI>(p, m, n0 + 8 * g, v, u);
}

template <class Mul, int EPI, int MB, int WAVES>
__global__ __launch_bounds__(64 * WAVES) void linear_block_kernel(const ArgsOf<EPI> p)
{
    constexpr int E = Mul::E, NB = EPI == EPI_GATED ? 2 : 1;
    constexpr int U = 4, TURN = 64 * U;                        // vectors per lane and turn, bytes of a row
    __shared__ __align__(16) f32x4 sums[WAVES][NB][MB][64];
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int r = lane & 15, group = lane >> 4;
    const int n0 = blockIdx.x * 16;
    const uint8_t* w[NB];
    const uint8_t* x[MB];
    w[0] = p.b + (int64_t)min(n0 + r, p.N - 1) * p.ldb;
    if constexpr (NB == 2) w[1] = p.b2 + (int64_t)min(n0 + r, p.N - 1) * p.ldb2;
#pragma unroll
    for (int i = 0; i < MB; ++i) x[i] = p.a + (int64_t)min(16 * i + r, p.M - 1) * p.lda;

    f32x4 acc[NB][MB];
#pragma unroll
    for (int j = 0; j < NB; ++j)
#pragma unroll
        for (int i = 0; i < MB; ++i) acc[j][i] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};

    const int64_t row = (int64_t)p.K * E;
    const int turns = (int)(row / TURN);
    u32x4 fw[2][NB][U], fx[2][MB][U];
    auto load = [&](int s, int turn) {
        const int64_t at = (int64_t)turn * TURN + 16 * group;
#pragma unroll
        for (int u = 0; u < U; ++u) {
#pragma unroll
            for (int j = 0; j < NB; ++j) __builtin_memcpy(&fw[s][j][u], w[j] + at + 64 * u, 16);
#pragma unroll
            for (int i = 0; i < MB; ++i) __builtin_memcpy(&fx[s][i][u], x[i] + at + 64 * u, 16);
        }
    };
    auto multiply = [&](int s) {
#pragma unroll
        for (int u = 0; u < U; ++u)
#pragma unroll
            for (int j = 0; j < NB; ++j)
#pragma unroll
                for (int i = 0; i < MB; ++i) acc[j][i] = Mul::mac16(fw[s][j][u], fx[s][i][u], acc[j][i]);
    };
    int t = wave;
    if (t < turns) load(0, t);
    while (t < turns) {
        if (t + WAVES < turns) load(1, t + WAVES);
        multiply(0);
        t += WAVES;
        if (t >= turns) break;
        if (t + WAVES < turns) load(0, t + WAVES);
        multiply(1);
        t += WAVES;
    }
    // the row's end goes to the wave whose turn it is
    if (t == turns && row > (int64_t)turns * TURN) {
        const int k0 = turns * (TURN / E) + group * (16 / E);
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int k = k0 + u * (64 / E);
#pragma unroll
            for (int j = 0; j < NB; ++j) fw[0][j][u] = load_piece<E>(w[j] + (int64_t)k * E, p.K - k);
#pragma unroll
            for (int i = 0; i < MB; ++i) fx[0][i][u] = load_piece<E>(x[i] + (int64_t)k * E, p.K - k);
        }
        multiply(0);
    }

#pragma unroll
    for (int j = 0; j < NB; ++j)
#pragma unroll
        for (int i = 0; i < MB; ++i) sums[wave][j][i][lane] = acc[j][i];
    __syncthreads();
    // value e of lane l is column 4 (l / 16) + e of row l % 16
    const int item = threadIdx.x;                              // row block, half of the columns, row
    if (item >= 32 * MB) return;
    const int i = item >> 5, half = item >> 4 & 1, m = item & 15;
    float v[8], u[8];
#pragma unroll
    for (int q = 0; q < 2; ++q) {
        f32x4 s[NB];
#pragma unroll
        for (int j = 0; j < NB; ++j) {
            s[j] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
            for (int y = 0; y < WAVES; ++y) s[j] += sums[y][j][i][m + 16 * (2 * half + q)];
        }
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            v[4 * q + e] = s[0][e];
            if constexpr (NB == 2) u[4 * q + e] = s[NB - 1][e];
        }
    }
    finish8<typename Mul::Out, EPI>(p, 16 * i + m, n0 + 8 * half, v, u);
}
// Eight waves a workgroup.  Where they take more than 128 registers (e4m3's widened operands, two row blocks) only one
// such workgroup runs on a CU, so past one a CU they come in fours: gated 9216 x 4096 on 16 rows in e4m3 22.9 -> 20.9 us,
// on 32 in bf16 49.9 -> 47.1; with fewer registers eight are faster (bf16 on four rows 33.5, in fours 34.7).
template <class Mul, int EPI, int MB> void launch_blocks(const ArgsOf<EPI>& p, int num_cu, hipStream_t stream)
{
    const int grid = (p.N + 15) / 16;
    if constexpr (Mul::E == 1 || MB == 2)
        if (grid > num_cu) {
            linear_block_kernel<Mul, EPI, MB, 4><<<grid, 256, 0, stream>>>(p);
            return;
        }
    linear_block_kernel<Mul, EPI, MB, 8><<<grid, 512, 0, stream>>>(p);
}

template <class Mul, int EPI> hipError_t launch_rows(const ProductArgs& args, int num_cu, hipStream_t stream)
{
    const auto& p = static_cast<const ArgsOf<EPI>&>(args);
    using Out = typename Mul::Out;
    constexpr int E = Mul::E, COLS = EPI == EPI_GATED ? WAVES : 2 * WAVES;
    const int rows_grid = (p.N + COLS - 1) / COLS;
    if (p.M <= 1) linear_few_kernel<E, Out, EPI, 1><<<rows_grid, 64 * WAVES, 0, stream>>>(p);
    else if (p.M <= vector_rows(E)) linear_few_kernel<E, Out, EPI, vector_rows(E)><<<rows_grid, 64 * WAVES, 0, stream>>>(p);
    else if (p.M <= 16) launch_blocks<Mul, EPI, 1>(p, num_cu, stream);
    else if (p.M <= FEW_ROWS) launch_blocks<Mul, EPI, 2>(p, num_cu, stream);
    else return hipErrorInvalidValue;
    return hipGetLastError();
}

template <class Mul> hipError_t launch_kind(Product kind, const ProductArgs& p, int num_cu, hipStream_t stream)
{
    if (kind == Product::FORWARD) return launch_rows<Mul, EPI_LINEAR>(p, num_cu, stream);
    if (kind == Product::GATED) return launch_rows<Mul, EPI_GATED>(p, num_cu, stream);
    if constexpr (Mul::E > 1)
        if (kind == Product::LOSS) return launch_rows<Mul, EPI_LOSS>(p, num_cu, stream);
    return hipErrorInvalidValue;
}

}  // namespace

hipError_t launch_product_few(Product kind, ProductType type, const ProductArgs& p, int num_cu, hipStream_t stream)
{
    switch (type) {
    case ProductType::BF16: return launch_kind<MulBf16>(kind, p, num_cu, stream);
    case ProductType::F32: return launch_kind<MulF32>(kind, p, num_cu, stream);
    // memory is the bound: the e4m3 instruction's short sums would gain nothing
    case ProductType::E4M3_BF16:
    case ProductType::E4M3_BF16_SHORT: return launch_kind<MulE4m3<Bf16, false>>(kind, p, num_cu, stream);
    case ProductType::E4M3_F32:
    case ProductType::E4M3_F32_SHORT: return launch_kind<MulE4m3<float, false>>(kind, p, num_cu, stream);
    case ProductType::BF16_F32:
        if (kind != Product::FORWARD) return hipErrorInvalidValue;
        return launch_rows<MulBf16F32, EPI_LINEAR>(p, num_cu, stream);
    }
    return hipErrorInvalidValue;
}

}  // namespace miconv
