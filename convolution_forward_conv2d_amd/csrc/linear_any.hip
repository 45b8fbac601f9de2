// linear_any.hip -- the product with its epilogue for any sizes, pitches and
// alignments: operands pass through registers on their way into LDS, so each
// 16-byte piece can be cut where a row or the reduction ends.
//
// Four waves, 2 x 2, on a tile of BM x BN; two LDS buffers, one barrier a
// step: the next step's pieces load into registers while the current step's
// products run.  It is for what the large tiles cannot take without a copy that
// costs more: small or unaligned products.  131 x 1001 x 4093
// in bf16 takes 12 us in ten parts and 4.5 to join them: the latency of its
// steps, one load to the next.
#include "linear_tile.h"
#include "kernels.h"

namespace miconv {

namespace {

constexpr int THREADS = 256;

// Raw B row j of a gated layer: the gate's or the other weights' row.
__device__ __forceinline__ int gated_row(int j, bool& up)
{
    up = (j & 16) != 0;
    return (j >> 5) * 16 + (j & 15);
}

template <int E, bool ACROSS, int R> struct Loader {
    static constexpr int N = R * 8 / THREADS;
    static constexpr int LINES = 128 / E;                      // k per step
    // rows [r0, ...) of `rows`, k from k0 of `K`
    template <bool GATED>
    __device__ static void load(u32x4 (&v)[N], const uint8_t* base, int64_t ld, const uint8_t* base2, int64_t ld2, int r0,
                                int rows, int k0, int K)
    {
#pragma unroll
        for (int i = 0; i < N; ++i) {
            const int q = threadIdx.x + i * THREADS;
            const int line = q >> 3, piece = q & 7;
            if constexpr (!ACROSS) {
                int r = r0 + line;
                const uint8_t* b = base;
                int64_t pitch = ld;
                if constexpr (GATED) {
                    bool up;
                    r = gated_row(r, up);
                    if (up) b = base2, pitch = ld2;
                }
                const int k = k0 + piece * (16 / E);
                v[i] = load_piece<E>(b + (int64_t)r * pitch + (int64_t)k * E, r < rows ? K - k : 0);
            } else {
                const int k = k0 + line % LINES;
                const int r = r0 + line / LINES * LINES + piece * (16 / E);
                v[i] = load_piece<E>(base + (int64_t)k * ld + (int64_t)r * E, k < K ? rows - r : 0);
            }
        }
    }
    __device__ static void store(const u32x4 (&v)[N], uint8_t* tile)
    {
#pragma unroll
        for (int i = 0; i < N; ++i) {
            const int q = threadIdx.x + i * THREADS;
            *reinterpret_cast<u32x4*>(tile + tile_piece<E, ACROSS>(q >> 3, q & 7)) = v[i];
        }
    }
};

template <class Mul, bool AACROSS, bool BACROSS, int EPI, int BM, int BN>
__global__ __launch_bounds__(THREADS) void linear_any_kernel(const ProductArgs p)
{
    constexpr int E = Mul::E, BK = 128 / E, FM = BM / 64, FN = BN / 64;
    constexpr int STEP = (BM + BN) * 128;
    constexpr int STAGE = 4 * 32 * (32 * FN + 4) * 4;
    __shared__ __align__(16) uint8_t smem[2 * STEP > STAGE ? 2 * STEP : STAGE];
    using LA = Loader<E, AACROSS, BM>;
    using LB = Loader<E, BACROSS, BN>;

    const int raw_n = EPI == EPI_GATED ? gated_raw_columns(p.N) : p.N;
    const int mt = (p.M + BM - 1) / BM, nt = (raw_n + BN - 1) / BN;
    int tm, tn;
    pick_tile(blockIdx.x, mt, nt, tm, tn);
    const int m0 = tm * BM, j0 = tn * BN;
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int wm = (wave >> 1) * 32 * FM, wn = (wave & 1) * 32 * FN;

    const int per_segment = (p.K + BK - 1) / BK;
    const int steps = per_segment * p.k_segments;
    const int first = (int)((int64_t)steps * blockIdx.z / p.splits);
    const int last = (int)((int64_t)steps * (blockIdx.z + 1) / p.splits);

    u32x4 va[LA::N], vb[LB::N];
    auto load = [&](int t) {
        const int seg = t >= per_segment;
        const int k = (t - seg * per_segment) * BK;
        // A's second segment starts k_pitch columns on; B's is another matrix
        const uint8_t* a = p.a + (int64_t)seg * p.k_pitch * (AACROSS ? p.lda : E);
        LA::template load<false>(va, a, p.lda, nullptr, 0, m0, p.M, k, p.K);
        const uint8_t* b = seg ? p.b2 : p.b;
        LB::template load<EPI == EPI_GATED>(vb, b, seg ? p.ldb2 : p.ldb, p.b2, p.ldb2, j0, p.N, k, p.K);
    };
    auto store = [&](int buf) {
        LA::store(va, smem + buf * STEP);
        LB::store(vb, smem + buf * STEP + BM * 128);
    };

    f32x16 acc[FM][FN];
#pragma unroll
    for (int i = 0; i < FM; ++i)
#pragma unroll
        for (int j = 0; j < FN; ++j)
#pragma unroll
            for (int e = 0; e < 16; ++e) acc[i][j][e] = 0.0f;

    if (first < last) {
        load(first);
        store(0);
    }
    __syncthreads();
    for (int t = first; t < last; ++t) {
        const int buf = (t - first) & 1;
        if (t + 1 < last) load(t + 1);
        const uint8_t* ta = smem + buf * STEP;
        const uint8_t* tb = ta + BM * 128;
#pragma unroll
        for (int s = 0; s < 2; ++s) {
            u32x4 fa[FM][2], fb[FN][2];
#pragma unroll
            for (int i = 0; i < FM; ++i) read_fragment<E, AACROSS>(ta, wm + 32 * i, s, lane, fa[i]);
#pragma unroll
            for (int j = 0; j < FN; ++j) read_fragment<E, BACROSS>(tb, wn + 32 * j, s, lane, fb[j]);
#pragma unroll
            for (int i = 0; i < FM; ++i)
#pragma unroll
                for (int j = 0; j < FN; ++j) acc[i][j] = Mul::mfma(fb[j], fa[i], acc[i][j]);
        }
        if (t + 1 < last) store(buf ^ 1);
        __syncthreads();
    }
    finish_wave<typename Mul::Out, EPI>(p, reinterpret_cast<float*>(smem) + wave * 32 * (32 * FN + 4), acc,
                                                m0 + wm, j0 + wn, blockIdx.z, lane);
}

template <class Mul, bool AACROSS, bool BACROSS, int EPI>
hipError_t launch_one(const ProductArgs& p, int tile, hipStream_t stream)
{
    const int raw_n = EPI == EPI_GATED ? gated_raw_columns(p.N) : p.N;
    const int64_t tiles = (int64_t)((p.M + tile - 1) / tile) * ((raw_n + tile - 1) / tile);
    if (tiles > INT32_MAX) return hipErrorInvalidValue;
    const dim3 grid((uint32_t)tiles, 1, (uint32_t)p.splits);
    if (tile == 128)
        linear_any_kernel<Mul, AACROSS, BACROSS, EPI, 128, 128><<<grid, THREADS, 0, stream>>>(p);
    else
        linear_any_kernel<Mul, AACROSS, BACROSS, EPI, 64, 64><<<grid, THREADS, 0, stream>>>(p);
    return hipGetLastError();
}

template <class Mul> hipError_t launch_type(Product kind, const ProductArgs& p, int tile, hipStream_t stream)
{
    switch (kind) {
    case Product::FORWARD: return launch_one<Mul, false, false, EPI_LINEAR>(p, tile, stream);
    case Product::GATED: return launch_one<Mul, false, false, EPI_GATED>(p, tile, stream);
    case Product::INPUT_GRAD: return launch_one<Mul, false, true, EPI_PLAIN>(p, tile, stream);
    case Product::WEIGHT_GRAD: return launch_one<Mul, true, true, EPI_PLAIN>(p, tile, stream);
    }
    return hipErrorInvalidValue;
}

template <class Mul> hipError_t launch_e4m3(Product kind, const ProductArgs& p, int tile, hipStream_t stream)
{
    if (kind == Product::FORWARD) return launch_one<Mul, false, false, EPI_LINEAR>(p, tile, stream);
    if (kind == Product::GATED) return launch_one<Mul, false, false, EPI_GATED>(p, tile, stream);
    return hipErrorInvalidValue;                               // no gradients in e4m3
}

template <class Out, int EPI>
__global__ __launch_bounds__(256) void join_kernel(const ProductArgs p)
{
    const int per = (p.N + 7) / 8;
    const int64_t total = (int64_t)p.M * per;
    for (int64_t it = blockIdx.x * 256ll + threadIdx.x; it < total; it += gridDim.x * 256ll) {
        const int m = (int)(it / per), n = (int)(it % per) * 8;
        const int raw = EPI == EPI_GATED ? (n >> 4) * 32 + (n & 15) : n;
        float v[8] = {}, u[8] = {};
#pragma unroll 4                                               // loads of four parts in flight together
        for (int z = 0; z < p.splits; ++z) {
            const float* at = p.part + ((int64_t)z * p.M + m) * p.part_ld + raw;
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const f32x4 x = reinterpret_cast<const f32x4*>(at)[h];
#pragma unroll
                for (int e = 0; e < 4; ++e) v[4 * h + e] += x[e];
                if constexpr (EPI == EPI_GATED) {
                    const f32x4 w = reinterpret_cast<const f32x4*>(at + 16)[h];
#pragma unroll
                    for (int e = 0; e < 4; ++e) u[4 * h + e] += w[e];
                }
            }
        }
        finish8<Out, EPI>(p, m, n, v, u);
    }
}

template <class Out> hipError_t join_type(Product kind, const ProductArgs& p, int blocks, hipStream_t stream)
{
    switch (kind) {
    case Product::FORWARD: join_kernel<Out, EPI_LINEAR><<<blocks, 256, 0, stream>>>(p); break;
    case Product::GATED: join_kernel<Out, EPI_GATED><<<blocks, 256, 0, stream>>>(p); break;
    default: join_kernel<Out, EPI_PLAIN><<<blocks, 256, 0, stream>>>(p); break;
    }
    return hipGetLastError();
}

}  // namespace

hipError_t launch_product_any(Product kind, ProductType type, const ProductArgs& p, int tile, hipStream_t stream)
{
    switch (type) {
    case ProductType::BF16: return launch_type<MulBf16>(kind, p, tile, stream);
    case ProductType::F32: return launch_type<MulF32>(kind, p, tile, stream);
    case ProductType::E4M3_BF16: return launch_e4m3<MulE4m3<Bf16, false>>(kind, p, tile, stream);
    case ProductType::E4M3_F32: return launch_e4m3<MulE4m3<float, false>>(kind, p, tile, stream);
    case ProductType::E4M3_BF16_SHORT: return launch_e4m3<MulE4m3<Bf16, true>>(kind, p, tile, stream);
    case ProductType::E4M3_F32_SHORT: return launch_e4m3<MulE4m3<float, true>>(kind, p, tile, stream);
    }
    return hipErrorInvalidValue;
}

hipError_t launch_product_join(Product kind, ProductType type, const ProductArgs& p, hipStream_t stream)
{
    const int64_t work = (int64_t)p.M * ((p.N + 7) / 8);
    const int blocks = (int)(work / 256 + 1 < 4096 ? work / 256 + 1 : 4096);
    if (type == ProductType::F32 || type == ProductType::E4M3_F32 || type == ProductType::E4M3_F32_SHORT)
        return join_type<float>(kind, p, blocks, stream);
    return join_type<Bf16>(kind, p, blocks, stream);
}

}  // namespace miconv
