// linear.cpp -- host side of the feed-forward operators: validation, the
// choice of kernel and tile, workspaces and launches.
#include <stdint.h>
#include <stdio.h>
#include <string.h>

#include <algorithm>

#include <hip/hip_runtime.h>

#include "miconv.h"
#include "handle.h"
#include "host_checks.h"
#include "linear_common.h"
#include "kernels.h"
#include "product.h"

namespace {

using namespace miconv;

bool valid_act(mic_activation a) { return (int)a >= 0 && (int)a <= (int)MIC_ACT_SILU; }

// Operands' rows (as they lie in memory) and their lengths in elements.
struct Extent {
    int a_rows, a_cols, b_rows, b_cols;
};

Extent extent_of(Product kind, int m, int n, int k)
{
    switch (kind) {
    case Product::INPUT_GRAD:
    case Product::INPUT_SUM: return {m, k, k, n};             // dz (m, k), w (k, n)
    case Product::WEIGHT_GRAD:
    case Product::CLASS_GRAD: return {k, m, k, n};            // dz (k, m), x (k, n)
    default: return {m, k, n, k};
    }
}

// The measured cost of a step (128 bytes of k) of each kernel's tile with every
// CU busy, microseconds, and of a tile's start and end; a launch; memory's rate
// for operands, copies and partial sums.  Only their ratios decide: 8192 x 8192
// outputs of 8192 terms take 754 us in four rounds of 256 x 256 and 859 in 5.4
// of 256 x 192; 4096 x 9216 of 4096 terms, 2.25 rounds of the one and exactly
// three of the other, 311 and 258.
constexpr double kReadPerUs = 4.5e6;
// A loss's blocks of few rows, which read whole rows of the weights, then end in their own rows' exponentials.  Measured,
// blocks and (128 x 256 tiles), us: 65536 x 4096 of 4 rows 103 (133), of 8 109 (133), of 16 137 (133); 50021 x 4096 of 8
// 88 (104); 128000 x 1024 of 4 64 (53), of 16 92 (50).
constexpr double kFewLossPerUs = 5.2e6, kFewLossRow = 0.12;
struct TileCost {
    int bm, bn;
    double step, tile;
};
constexpr TileCost kFast[] = {{256, 256, 1.50, 3.0}, {256, 192, 1.12, 3.0}, {192, 256, 1.12, 3.0}, {256, 128, 0.87, 2.5},
                              {128, 256, 0.93, 2.5}, {128, 128, 0.47, 2.5}, {128, 64, 0.0, 2.0},  {64, 128, 0.0, 2.0}};
constexpr double kF32Step = 1.9;                       // 128 x 128 in fp32; of the smaller tiles, its share

// linear_few.hip's blocks: their start, then memory's time for the weights or a CU's for its workgroups' weights and x, about
// 37 KB a microsecond (a third of it where rows are not 16-byte aligned).  Measured, with the tiles' time behind it:
// 16 rows of 1000 x 4096 9.7 us (13.2), of 2048 x 2048 gated 8.4 (12.4), 32 of 4096 x 9216 27.0 (25), of 4001 x 4093
// 29.2 (20.3).
double few_us(int num_cu, int m, int raw_n, bool gated, double row_bytes, bool aligned)
{
    const int columns = gated ? 32 : 16;
    const double groups = std::max(1.0, (double)raw_n / columns / num_cu), rate = aligned ? 37.0e3 : 15.0e3;
    const double x_rows = (m + 15) / 16 * 16;
    return 2.5 + std::max(raw_n * row_bytes / kReadPerUs, groups * (columns + x_rows) * row_bytes / rate);
}

}  // namespace

namespace miconv {

// The cheapest way through a product of m x n outputs and k_segments * k terms.
// `aligned_a` / `aligned_b`: the operand's rows can be read 16 bytes at a time.
Plan plan_product(int num_cu, Product kind, ProductType type, int m, int n, int k, int k_segments, bool aligned_a,
                  bool aligned_b, int least_splits)
{
    // a loss's epilogues need whole sums, in large tiles or few rows
    const bool whole = kind == Product::LOSS || kind == Product::LOGITS_GRAD;
    const bool of_loss = kind >= Product::LOSS || type == ProductType::BF16_F32;
    const int raw_n = kind == Product::GATED ? miconv::gated_raw_columns(n) : n;
    const int e = element_bytes(type);
    const int64_t steps = (int64_t)((k + 128 / e - 1) / (128 / e)) * k_segments;
    auto tiles = [&](int bm, int bn) { return (int64_t)((m + bm - 1) / bm) * ((raw_n + bn - 1) / bn); };
    // a reduction is split where tiles leave CUs idle: parts of at least four steps, no more than fill the CUs twice
    auto most_splits = [&](int64_t t) {
        return (int)std::max<int64_t>(1, std::min<int64_t>({2 * num_cu / std::max<int64_t>(t, 1), steps / 4, 32}));
    };
    auto join_us = [&](int splits) {
        return splits > 1 ? kLaunchUs + (double)m * raw_n * 4 * 2 * splits / kBytesPerUs : 0.0;
    };
    auto rounds = [&](int64_t t, int slots) { return (double)((t + slots - 1) / slots); };
    const double b_bytes = (double)raw_n * k * k_segments * e, read_us = (b_bytes + (double)m * k * k_segments * e) / kReadPerUs;
    Plan best = {};
    best.us = 1e30;
    // (a loss of more classes than a grid of 16 to a workgroup reaches goes on tiles)
    const bool few_loss = kind == Product::LOSS && n < 1 << 26;
    if (m <= miconv::FEW_ROWS && (kind == Product::FORWARD || kind == Product::GATED || few_loss)) {
        best.few = true;
        best.splits = 1;
        // one or two rows on the vector units: faster at every size and alignment measured (4001 x 4093, rows of odd
        // lengths, 11.4 us against 22.0)
        if (m <= miconv::vector_rows(e)) {
            best.us = 0.0;
            return best;
        }
        best.us = few_us(num_cu, m, raw_n, kind == Product::GATED, (double)k * e, aligned_a && aligned_b);
        if (kind == Product::LOSS && e == 2 && aligned_a && aligned_b)
            best.us = 2.5 + b_bytes / kFewLossPerUs + kFewLossRow * m * std::max(1.0, (double)n / 16 / num_cu);
    }
    auto consider = [&](Plan pl, int64_t t, int bm, int bn, int slots, double step, double tile) {
        // HIP takes grids of fewer than 2^32 threads: 2^30 rows of 64 x 64 are past that
        if (t * (pl.fast ? 512 : 256) >= int64_t(1) << 32) return;
        // weights that one or two row tiles read come from memory at its latency, two steps in flight; a loss's products
        // price it by the tile: a CU takes about 46 KB a microsecond, and a step 0.72 (256 x 4096 of 1000 terms, dx of a
        // small classifier: 256 x 128 18.5 us, 128 x 128 and 64 x 64 14)
        if (m <= 2 * bm) step = std::max(step, of_loss ? std::max(0.72, (bm + bn) * 128 / 46.0e3) : 0.9);
        const int most = whole ? 1 : std::max(least_splits, most_splits(t));
        for (int s = least_splits; s <= most; ++s) {
            const double busy = rounds(t * s, slots) * ((steps + s - 1) / s * step + tile);
            double us = std::max(busy, read_us) + join_us(s) + pl.us + 1.5;
            // of tiles that all wait for memory, the one that does less beside it
            if (of_loss) us += 0.05 * std::min(busy, read_us);
            if (us < best.us) {
                best = pl;
                best.splits = s;
                best.us = us;
                best.part_ld = align_up(raw_n, bn);
            }
        }
    };
    // linear_any.hip: two workgroups per CU on 128 x 128 tiles, four on 64 x 64; fp32's matrix instructions take
    // sixteen times bf16's time for the same bytes
    const double slow = type == ProductType::F32 ? 4.0 : element_bytes(type) == 2 ? 1.0 : 1.2;
    Plan any = {};
    any.tile = 128;
    if (!whole) consider(any, tiles(128, 128), 128, 128, 2 * num_cu, 1.45 * slow, 2.0);
    any.tile = 64;
    if (!whole) consider(any, tiles(64, 64), 64, 64, 4 * num_cu, 1.10 * slow, 1.5);

    const Extent x = extent_of(kind, m, n, k);
    const bool short_rows = (int64_t)std::max(x.a_cols, x.b_cols) * e < kMaxPitchBytes / 2 - 64;
    // two k segments are one matrix, laid out by the library and aligned
    const bool f32 = type == ProductType::F32;
    // a step's 128 bytes are twice the products in e4m3, which only its own instruction takes in bf16's time
    const double widened = type == ProductType::E4M3_BF16 || type == ProductType::E4M3_F32 ? 2.0 : 1.0;
    if (short_rows && (aligned_a || k_segments == 1)) {
        Plan pl = {};
        pl.fast = true;
        if (!aligned_a) {
            pl.pack_a = align_up((int64_t)x.a_cols * e, 16);
            pl.a_bytes = (size_t)align_up(pl.pack_a * x.a_rows, 256);
            pl.us += 2.0 * pl.a_bytes / kBytesPerUs;
        }
        if (!aligned_b) {
            const int copies = kind == Product::GATED ? 2 : k_segments;
            pl.pack_b = align_up((int64_t)x.b_cols * e, 16);
            pl.b_bytes = (size_t)align_up(pl.pack_b * x.b_rows, 256);
            pl.us += copies * 2.0 * pl.b_bytes / kBytesPerUs;
        }
        if (pl.pack_a || pl.pack_b) pl.us += kLaunchUs;
        for (int i = 0; i < (int)miconv::FastTile::COUNT; ++i) {
            const TileCost& c = kFast[i];
            pl.fast_tile = (miconv::FastTile)i;
            const bool small = c.bm * c.bn <= 128 * 128;
            if (f32 && small)
                consider(pl, tiles(c.bm, c.bn), c.bm, c.bn, num_cu, kF32Step * c.bm * c.bn / (128 * 128), c.tile);
            else if (!f32 && c.step > 0) {
                // many rounds of a loss's tiles: 4096 x 50021 of 4096 terms take 1321 us in 12.25 rounds of 256 x 256
                // and 1364 in 16.3 of 256 x 192.  192 x 256 costs the same: priced at 1.12, it took 48 sizes over that
                // it should not have, 1.8 percent slower in all (618 x 80049 of 3848 terms 423 -> 478 us, 1351 x 55441
                // of 2768 389 -> 434; others within 2 percent)
                const double step = whole && c.bm * c.bn == 256 * 192 ? 1.18 : c.step;
                consider(pl, tiles(c.bm, c.bn), c.bm, c.bn, num_cu, step * widened, c.tile);
            }
        }
    }
    const int copies = kind == Product::GATED ? 2 : k_segments;
    best.bytes = best.a_bytes + copies * best.b_bytes
                 + (best.splits > 1 ? (size_t)best.splits * m * best.part_ld * 4 : 0);
    return best;
}

void describe(const Plan& pl, char* text, size_t size)
{
    constexpr const char* kFastNames[] = {"256x256", "256x192", "192x256", "256x128", "128x256", "128x128", "128x64", "64x128"};
    static_assert(sizeof(kFastNames) / sizeof(*kFastNames) == (size_t)miconv::FastTile::COUNT, "one name a tile");
    int at;
    if (pl.few) at = snprintf(text, size, "few");
    else if (pl.fast) at = snprintf(text, size, "fast %s", kFastNames[(int)pl.fast_tile]);
    else at = snprintf(text, size, "any %dx%d", pl.tile, pl.tile);
    if (pl.splits > 1) at += snprintf(text + at, size - at, " split %d", pl.splits);
    if (pl.pack_a) at += snprintf(text + at, size - at, " pack a");
    if (pl.pack_b) snprintf(text + at, size - at, " pack b");
}

static bool fast_rows(const uint8_t* p, int64_t ld, int64_t bytes) { return aligned_matrix(p, ld) && bytes % 16 == 0; }

// The lengths a product's operands are padded to, where the caller has not said more.
static void fill(ProductArgs& p)
{
    if (p.a_K < p.K) p.a_K = p.K;
    if (p.a_rows < p.M) p.a_rows = p.M;
    if (p.b_rows < p.N) p.b_rows = p.N;
}

mic_status run_pair(mic_handle h, ProductType type, ProductArgs& dx, ProductArgs& dw)
{
    fill(dx);
    fill(dw);
    return launched(launch_product_pair(type, dx, dw, h->stream));
}

mic_status run_product(mic_handle h, Product kind, ProductType type, ProductArgs& p, void* workspace, size_t bytes, Sums* sums)
{
    if (p.M == 0 || p.N == 0) return MIC_STATUS_SUCCESS;
    const int e = element_bytes(type);
    const bool a_across = kind == Product::WEIGHT_GRAD || kind == Product::CLASS_GRAD;
    const bool b_across = a_across || kind == Product::INPUT_GRAD || kind == Product::INPUT_SUM;
    fill(p);
    const bool two_b = kind == Product::GATED || p.k_segments > 1;
    bool aligned_a = fast_rows(p.a, p.lda, (int64_t)(a_across ? p.a_rows : p.a_K) * e);
    const int64_t b_bytes = (int64_t)(b_across ? p.b_rows : p.a_K) * e;
    bool aligned_b = fast_rows(p.b, p.ldb, b_bytes);
    if (two_b) aligned_b = aligned_b && fast_rows(p.b2, p.ldb2, b_bytes);
    if (p.k_segments > 1) aligned_b = aligned_b && p.ldb == p.ldb2;
    const Plan pl = plan_product(h->num_cu, kind, type, p.M, p.N, p.K, p.k_segments, aligned_a, aligned_b, p.splits > 1 ? p.splits : 1);
    if (!planned(pl)) return MIC_STATUS_NOT_SUPPORTED;
    if (pl.bytes > bytes || (pl.bytes && (!workspace || !aligned(workspace, 16)))) return MIC_STATUS_BAD_PARAM;
    uint8_t* ws = static_cast<uint8_t*>(workspace);
    const Extent x = extent_of(kind, p.M, p.N, p.K);
    miconv::PackJob jobs[miconv::PACK_JOBS];
    int packs = 0;
    auto pack = [&](const uint8_t*& from, int64_t& ld, int64_t rows, int64_t bytes, int64_t pitch, size_t size) {
        jobs[packs++] = {from, ld, rows, bytes, ws, pitch};
        from = ws, ld = pitch;
        ws += size;
    };
    if (pl.pack_a) {
        pack(p.a, p.lda, x.a_rows, (int64_t)x.a_cols * e, pl.pack_a, pl.a_bytes);
        if (a_across) p.a_rows = (int)(pl.pack_a / e);
    }
    if (pl.pack_b) {
        pack(p.b, p.ldb, x.b_rows, (int64_t)x.b_cols * e, pl.pack_b, pl.b_bytes);
        if (two_b) pack(p.b2, p.ldb2, x.b_rows, (int64_t)x.b_cols * e, pl.pack_b, pl.b_bytes);
        if (b_across) p.b_rows = (int)(pl.pack_b / e);
    }
    if (packs) MIC_TRY(launched(miconv::launch_pack(jobs, packs, h->stream)));
    p.splits = pl.splits;
    p.part = reinterpret_cast<float*>(ws);
    p.part_ld = pl.part_ld;
    hipError_t err = pl.few    ? miconv::launch_product_few(kind, type, p, h->num_cu, h->stream)
                     : pl.fast ? miconv::launch_product_fast(kind, type, p, pl.fast_tile, h->stream)
                               : miconv::launch_product_any(kind, type, p, pl.tile, h->stream);
    if (sums) *sums = pl.splits > 1 ? Sums{p.part, p.part_ld, pl.splits} : Sums{static_cast<const float*>(p.y), p.ldy, 1};
    if (err == hipSuccess && pl.splits > 1 && !sums) err = miconv::launch_product_join(kind, type, p, h->stream);
    return launched(err);
}

}  // namespace miconv

namespace {

// Workspace for any alignment of the operands.
size_t product_bytes(int num_cu, Product kind, ProductType type, int m, int n, int k, int k_segments)
{
    if (!m || !n) return 0;
    size_t most = 0;
    for (int a = 0; a < 2; ++a)
        for (int b = 0; b < 2; ++b)
            most = std::max(most, plan_product(num_cu, kind, type, m, n, k, k_segments, a != 0, b != 0).bytes);
    return most;
}

// Which of a product's operands can be read 16 bytes at a time, where the caller says that every operand's pointer and
// pitch is a multiple of 16 bytes (`aligned`).  A gradient's dz is the library's own (`own_dz`) unless it is dy.
struct Aligned {
    bool a, b;
};

Aligned aligned_operands(Product kind, ProductType type, int n, int k, bool aligned, bool own_dz, int64_t dz_pitch)
{
    const int e = element_bytes(type);
    auto even = [&](int64_t cols) { return cols * e % 16 == 0 && cols * e < kMaxPitchBytes / 2; };
    const bool x = aligned && even(k);                         // x's rows and w's are k long
    if (kind == Product::FORWARD || kind == Product::GATED) return {x, x};
    return {own_dz ? even(dz_pitch) : aligned && even(n), x};
}

// The same for operands of known alignment.
size_t aligned_bytes(int num_cu, Product kind, ProductType type, int m, int n, int k, int k_segments, Aligned al)
{
    return m && n ? plan_product(num_cu, kind, type, m, n, k, k_segments, al.a, al.b).bytes : 0;
}

mic_status product_type(mic_dtype in, mic_dtype out, ProductType* type, bool fast = false)
{
    if (in == MIC_DTYPE_F32 && out == MIC_DTYPE_F32) *type = ProductType::F32;
    else if (in == MIC_DTYPE_BF16 && out == MIC_DTYPE_BF16) *type = ProductType::BF16;
    else if (in == MIC_DTYPE_F8_E4M3 && out == MIC_DTYPE_BF16) *type = fast ? ProductType::E4M3_BF16_SHORT : ProductType::E4M3_BF16;
    else if (in == MIC_DTYPE_F8_E4M3 && out == MIC_DTYPE_F32) *type = fast ? ProductType::E4M3_F32_SHORT : ProductType::E4M3_F32;
    else return MIC_STATUS_NOT_SUPPORTED;
    return MIC_STATUS_SUCCESS;
}

mic_status forward_workspace(mic_handle h, Product kind, mic_dtype dtype, int m, int n, int k, bool aligned, size_t* bytes)
{
    if (!bytes) return MIC_STATUS_BAD_PARAM;
    MIC_TRY(check_sizes(m, n, k));
    if (kind == Product::GATED && n >= kMaxSize / 2) return MIC_STATUS_NOT_SUPPORTED;      // twice as many raw columns
    ProductType type, fast;
    MIC_TRY(product_type(dtype, plain_type(dtype) ? dtype : MIC_DTYPE_BF16, &type));
    MIC_TRY(product_type(dtype, plain_type(dtype) ? dtype : MIC_DTYPE_BF16, &fast, true));
    *bytes = most_bytes(h, [&](int cus) {
        auto need = [&](ProductType t) {
            if (!aligned) return product_bytes(cus, kind, t, m, n, k, 1);
            return aligned_bytes(cus, kind, t, m, n, k, 1, aligned_operands(kind, t, n, k, true, false, 0));
        };
        return std::max(need(type), need(fast));
    });
    return MIC_STATUS_SUCCESS;
}

mic_status forward_name(mic_handle h, Product kind, mic_dtype dtype, mic_dtype out_dtype, int fast_sums, int m, int n, int k,
                        int aligned, char* buf, size_t buflen)
{
    MIC_TRY(check_sizes(m, n, k));
    if (kind == Product::GATED && n >= kMaxSize / 2) return MIC_STATUS_NOT_SUPPORTED;
    ProductType type;
    MIC_TRY(product_type(dtype, out_dtype, &type, fast_sums != 0));
    if (!m || !n) return give_name("nothing", buf, buflen);
    const Aligned al = aligned_operands(kind, type, n, k, aligned != 0, false, 0);
    const Plan pl = plan_product(cus_of(h), kind, type, m, n, k, 1, al.a, al.b);
    if (!planned(pl)) return MIC_STATUS_NOT_SUPPORTED;
    char text[64];
    describe(pl, text, sizeof(text));
    return give_name(text, buf, buflen);
}

// The backward workspace: dz, dbias's partial sums, the products' own.
struct GradLayout {
    int64_t pitch;           // of one layer's dz columns
    size_t dz, sums, product, total;
};

// `aligned`: every operand is; without an activation (own_dz false) dz is then dy, read where it is and never copied.
GradLayout grad_layout(int num_cu, ProductType type, int m, int n, int k, bool gated, bool bias, bool aligned, bool own_dz)
{
    GradLayout g = {};
    const int two = gated ? 2 : 1;
    g.pitch = align_up(n, 64);
    if (own_dz) g.dz = (size_t)align_up((int64_t)m * g.pitch * two * (type == ProductType::F32 ? 4 : 2), 256);
    g.sums = bias ? (size_t)align_up((int64_t)miconv::slope_row_groups(m, n) * n * 4, 256) : 0;
    const int wide = (int)(gated ? 2 * g.pitch : n);
    if (aligned) {
        auto bytes = [&](Product kind, int rows, int columns, int terms, int segments) {
            return aligned_bytes(num_cu, kind, type, rows, columns, terms, segments,
                                 aligned_operands(kind, type, n, k, true, own_dz, two * g.pitch));
        };
        g.product = std::max(bytes(Product::INPUT_GRAD, m, k, n, two), bytes(Product::WEIGHT_GRAD, wide, k, m, 1));
    } else {
        g.product = std::max(product_bytes(num_cu, Product::INPUT_GRAD, type, m, k, n, two),
                             product_bytes(num_cu, Product::WEIGHT_GRAD, type, wide, k, m, 1));
    }
    g.total = g.dz + g.sums + g.product;
    return g;
}

mic_status backward_workspace(mic_handle h, mic_dtype dtype, int m, int n, int k, bool gated, bool aligned, bool own_dz,
                              size_t* bytes)
{
    if (!bytes) return MIC_STATUS_BAD_PARAM;
    MIC_TRY(check_sizes(m, n, k));
    if (!plain_type(dtype)) return MIC_STATUS_NOT_SUPPORTED;
    if (n >= kMaxSize / 2) return MIC_STATUS_NOT_SUPPORTED;
    ProductType type;
    MIC_TRY(product_type(dtype, dtype, &type));
    *bytes = most_bytes(h, [&](int cus) { return grad_layout(cus, type, m, n, k, gated, !gated, aligned, own_dz).total; });
    return MIC_STATUS_SUCCESS;
}

mic_status backward_name(mic_handle h, mic_dtype dtype, bool own_dz, int m, int n, int k, bool gated, int aligned, char* buf,
                         size_t buflen)
{
    MIC_TRY(check_sizes(m, n, k));
    if (!plain_type(dtype)) return MIC_STATUS_NOT_SUPPORTED;
    if (n >= kMaxSize / 2) return MIC_STATUS_NOT_SUPPORTED;
    ProductType type;
    MIC_TRY(product_type(dtype, dtype, &type));
    if (!k) return give_name("nothing", buf, buflen);
    const int two = gated ? 2 : 1;
    const int64_t pitch = align_up(n, 64);
    char dx[64] = "nothing", dw[64] = "nothing", text[160];
    if (m) {
        const Aligned al = aligned_operands(Product::INPUT_GRAD, type, n, k, aligned != 0, own_dz, two * pitch);
        const Plan pl = plan_product(cus_of(h), Product::INPUT_GRAD, type, m, k, n, two, al.a, al.b);
        if (!planned(pl)) return MIC_STATUS_NOT_SUPPORTED;
        describe(pl, dx, sizeof(dx));
    }
    if (n) {
        const Aligned al = aligned_operands(Product::WEIGHT_GRAD, type, n, k, aligned != 0, own_dz, two * pitch);
        const Plan pl = plan_product(cus_of(h), Product::WEIGHT_GRAD, type, gated ? (int)(2 * pitch) : n, k, m, 1, al.a, al.b);
        if (!planned(pl)) return MIC_STATUS_NOT_SUPPORTED;
        describe(pl, dw, sizeof(dw));
    }
    snprintf(text, sizeof(text), "dx: %s, dw: %s", dx, dw);
    return give_name(text, buf, buflen);
}

// dx = dz w (+ dz2 w2) and dw = dz^T x (dw2 = dz2^T x).  dz has dz_cols >= n columns, zeros from n on (and the
// second layer's from up_at on).
mic_status grad_products(mic_handle h, ProductType type, int m, int n, int k, const void* dz, int64_t dz_pitch,
                         int64_t dz_cols, int64_t up_at, const void* x, int64_t ldx, const void* w, int64_t ldw, const void* w2,
                         int64_t ldw2, void* dx, int64_t lddx, void* dw, int64_t lddw, void* dw2, int64_t lddw2,
                         void* workspace, size_t bytes)
{
    const int64_t e = type == ProductType::F32 ? 4 : 2;
    const bool gated = w2 != nullptr || dw2 != nullptr;
    if (dx) {
        ProductArgs p = {};
        p.a = static_cast<const uint8_t*>(dz), p.lda = dz_pitch * e;
        p.b = static_cast<const uint8_t*>(w), p.ldb = ldw * e;
        p.b2 = static_cast<const uint8_t*>(w2), p.ldb2 = ldw2 * e;
        p.M = m, p.N = k, p.K = n, p.a_K = (int)dz_cols;
        p.k_segments = gated ? 2 : 1, p.k_pitch = (int)up_at;
        p.m_pitch = INT32_MAX, p.m_valid = m;
        p.y = dx, p.ldy = lddx;
        MIC_TRY(run_product(h, Product::INPUT_GRAD, type, p, workspace, bytes));
    }
    if (dw) {
        ProductArgs p = {};
        p.a = static_cast<const uint8_t*>(dz), p.lda = dz_pitch * e;
        p.b = static_cast<const uint8_t*>(x), p.ldb = ldx * e;
        p.M = gated ? (int)(2 * up_at) : n, p.N = k, p.K = m, p.a_rows = gated ? p.M : (int)dz_cols;
        p.k_segments = 1;
        p.m_pitch = gated ? (int)up_at : INT32_MAX, p.m_valid = n;
        p.y = dw, p.ldy = lddw;
        p.y2 = dw2, p.ldy2 = lddw2;
        MIC_TRY(run_product(h, Product::WEIGHT_GRAD, type, p, workspace, bytes));
    }
    return MIC_STATUS_SUCCESS;
}

}  // namespace

extern "C" {

mic_status mic_rms_norm(mic_handle handle, mic_dtype dtype, mic_dtype out_dtype, int rows, int cols, double eps,
                        const void* x, int64_t ldx, const void* residual, int64_t ldr, const void* weight,
                        void* y, int64_t ldy, void* sum, int64_t lds, float* rstd, float* scale)
{
    if (!handle) return MIC_STATUS_BAD_PARAM;
    if (!plain_type(dtype) || (out_dtype != dtype && out_dtype != MIC_DTYPE_F8_E4M3)) return MIC_STATUS_NOT_SUPPORTED;
    MIC_TRY(check_sizes(rows, cols, 0));
    if (!(eps >= 0.0)) return MIC_STATUS_BAD_PARAM;
    if (rows == 0) return MIC_STATUS_SUCCESS;
    if (cols == 0) return MIC_STATUS_BAD_PARAM;                // the mean of nothing
    const size_t e = size_of(dtype);
    const bool e4m3 = out_dtype == MIC_DTYPE_F8_E4M3;
    MIC_TRY(check_matrix(x, ldx, rows, cols, e));
    if (residual) MIC_TRY(check_matrix(residual, ldr, rows, cols, e));
    if (sum) MIC_TRY(check_matrix(sum, lds, rows, cols, e));
    MIC_TRY(check_matrix(y, ldy, rows, cols, size_of(out_dtype)));
    if (!weight || !aligned(weight, e) || !aligned(rstd, 4) || !aligned(scale, 4)) return MIC_STATUS_BAD_PARAM;
    if (e4m3 && !scale) return MIC_STATUS_BAD_PARAM;
    miconv::NormArgs p = {rows, cols, (float)eps, x, ldx, residual, ldr, weight, y, ldy, sum, lds, rstd, scale};
    return launched(miconv::launch_rms_norm(device_type(dtype), e4m3, p, handle->stream));
}

mic_status mic_rms_norm_backward_workspace(mic_handle handle, int rows, int cols, size_t* bytes)
{
    if (!bytes) return MIC_STATUS_BAD_PARAM;
    MIC_TRY(check_sizes(rows, cols, 0));
    *bytes = most_bytes(handle, [&](int cus) { return (size_t)miconv::rms_norm_grad_groups(rows, cols, cus) * cols * 4; });
    return MIC_STATUS_SUCCESS;
}

mic_status mic_rms_norm_backward(mic_handle handle, mic_dtype dtype, int rows, int cols, const void* dy, int64_t lddy,
                                 const void* sum, int64_t lds, const void* weight, const float* rstd,
                                 const void* dsum, int64_t ldd, void* dx, int64_t lddx, void* dweight,
                                 void* workspace, size_t workspace_bytes)
{
    if (!handle) return MIC_STATUS_BAD_PARAM;
    if (!plain_type(dtype)) return MIC_STATUS_NOT_SUPPORTED;
    size_t need;
    MIC_TRY(mic_rms_norm_backward_workspace(handle, rows, cols, &need));
    if (cols == 0) return rows == 0 ? MIC_STATUS_SUCCESS : MIC_STATUS_BAD_PARAM;
    const size_t e = size_of(dtype);
    MIC_TRY(check_matrix(dy, lddy, rows, cols, e));
    MIC_TRY(check_matrix(sum, lds, rows, cols, e));
    if (dsum) MIC_TRY(check_matrix(dsum, ldd, rows, cols, e));
    MIC_TRY(check_matrix(dx, lddx, rows, cols, e));
    if (!weight || !aligned(weight, e) || !aligned(dweight, e)) return MIC_STATUS_BAD_PARAM;
    if (rows && (!rstd || !aligned(rstd, 4))) return MIC_STATUS_BAD_PARAM;
    if (rows == 0 && !dweight) return MIC_STATUS_SUCCESS;
    if (dweight && (!workspace || !aligned(workspace, 16) || workspace_bytes < need)) return MIC_STATUS_BAD_PARAM;
    miconv::NormGradArgs p = {rows, cols, dy, lddy, sum, lds, weight, rstd, dsum, ldd, dx, lddx, dweight,
                              static_cast<float*>(workspace),
                              miconv::rms_norm_grad_groups(rows, cols, handle->num_cu)};
    return launched(miconv::launch_rms_norm_grad(device_type(dtype), p, handle->stream));
}

mic_status mic_linear_forward_workspace(mic_handle handle, mic_dtype dtype, int m, int n, int k, size_t* bytes)
{
    return forward_workspace(handle, Product::FORWARD, dtype, m, n, k, false, bytes);
}

mic_status mic_linear_forward_workspace_aligned(mic_handle handle, mic_dtype dtype, int m, int n, int k, size_t* bytes)
{
    return forward_workspace(handle, Product::FORWARD, dtype, m, n, k, true, bytes);
}

mic_status mic_linear_forward(mic_handle handle, mic_dtype dtype, mic_dtype out_dtype, mic_activation act,
                              int fast_sums, int m, int n, int k, const void* x, int64_t ldx, const void* w, int64_t ldw,
                              const float* x_scale, const float* w_scale, const void* bias, const void* residual,
                              int64_t ldr, void* y, int64_t ldy, void* preact, int64_t ldp, void* workspace,
                              size_t workspace_bytes)
{
    if (!handle) return MIC_STATUS_BAD_PARAM;
    ProductType type;
    MIC_TRY(product_type(dtype, out_dtype, &type, fast_sums != 0));
    if (!valid_act(act)) return MIC_STATUS_NOT_SUPPORTED;
    MIC_TRY(check_sizes(m, n, k));
    if (m == 0 || n == 0) return MIC_STATUS_SUCCESS;
    const size_t e = size_of(dtype), o = size_of(out_dtype);
    MIC_TRY(check_matrix(x, ldx, m, k, e));
    MIC_TRY(check_matrix(w, ldw, n, k, e));
    MIC_TRY(check_matrix(y, ldy, m, n, o));
    if (residual) MIC_TRY(check_matrix(residual, ldr, m, n, o));
    if (preact) MIC_TRY(check_matrix(preact, ldp, m, n, o));
    if (!aligned(bias, o) || !aligned(x_scale, 4) || !aligned(w_scale, 4)) return MIC_STATUS_BAD_PARAM;
    const bool scaled = dtype == MIC_DTYPE_F8_E4M3;
    if (scaled != (x_scale != nullptr) || scaled != (w_scale != nullptr)) return MIC_STATUS_BAD_PARAM;
    ProductArgs p = {};
    p.a = static_cast<const uint8_t*>(x), p.lda = ldx * (int64_t)e;
    p.b = static_cast<const uint8_t*>(w), p.ldb = ldw * (int64_t)e;
    p.M = m, p.N = n, p.K = k, p.k_segments = 1;
    p.act = act;
    p.y = y, p.ldy = ldy;
    p.bias = bias, p.residual = residual, p.ldr = ldr;
    p.x_scale = x_scale, p.w_scale = w_scale;
    p.pre = preact, p.ldp = ldp;
    return run_product(handle, Product::FORWARD, type, p, workspace, workspace_bytes);
}

mic_status mic_linear_forward_kernel_name(mic_handle handle, mic_dtype dtype, mic_dtype out_dtype, int fast_sums, int m,
                                          int n, int k, int aligned, char* buf, size_t buflen)
{
    return forward_name(handle, Product::FORWARD, dtype, out_dtype, fast_sums, m, n, k, aligned, buf, buflen);
}

mic_status mic_gated_linear_forward_kernel_name(mic_handle handle, mic_dtype dtype, mic_dtype out_dtype, int fast_sums,
                                                int m, int n, int k, int aligned, char* buf, size_t buflen)
{
    return forward_name(handle, Product::GATED, dtype, out_dtype, fast_sums, m, n, k, aligned, buf, buflen);
}

mic_status mic_linear_backward_kernel_name(mic_handle handle, mic_dtype dtype, mic_activation act, int m, int n, int k,
                                           int aligned, char* buf, size_t buflen)
{
    if (!valid_act(act)) return MIC_STATUS_NOT_SUPPORTED;
    return backward_name(handle, dtype, act != MIC_ACT_NONE, m, n, k, false, aligned, buf, buflen);
}

mic_status mic_gated_linear_backward_kernel_name(mic_handle handle, mic_dtype dtype, int m, int n, int k, int aligned,
                                                 char* buf, size_t buflen)
{
    return backward_name(handle, dtype, true, m, n, k, true, aligned, buf, buflen);
}

mic_status mic_linear_backward_workspace(mic_handle handle, mic_dtype dtype, int m, int n, int k, size_t* bytes)
{
    return backward_workspace(handle, dtype, m, n, k, false, false, true, bytes);
}

mic_status mic_linear_backward_workspace_aligned(mic_handle handle, mic_dtype dtype, mic_activation act, int m, int n, int k,
                                                 size_t* bytes)
{
    if (!valid_act(act)) return MIC_STATUS_NOT_SUPPORTED;
    return backward_workspace(handle, dtype, m, n, k, false, true, act != MIC_ACT_NONE, bytes);
}

mic_status mic_linear_backward(mic_handle handle, mic_dtype dtype, mic_activation act, int m, int n, int k,
                               const void* dy, int64_t lddy, const void* x, int64_t ldx, const void* w, int64_t ldw,
                               const void* preact, int64_t ldp, void* dx, int64_t lddx, void* dw, int64_t lddw,
                               void* dbias, void* workspace, size_t workspace_bytes)
{
    if (!handle) return MIC_STATUS_BAD_PARAM;
    const size_t e = size_of(dtype);
    const bool slope = act != MIC_ACT_NONE;
    const bool even = (!dw || aligned_matrix(x, ldx * (int64_t)e)) && (!dx || aligned_matrix(w, ldw * (int64_t)e))
                      && (slope || aligned_matrix(dy, lddy * (int64_t)e));
    size_t need;
    MIC_TRY(backward_workspace(handle, dtype, m, n, k, false, even, slope || !even, &need));
    if (!valid_act(act)) return MIC_STATUS_NOT_SUPPORTED;
    MIC_TRY(check_matrix(dy, lddy, m, n, e));
    if (slope) MIC_TRY(check_matrix(preact, ldp, m, n, e));
    if (dw) MIC_TRY(check_matrix(x, ldx, m, k, e));
    if (dx) MIC_TRY(check_matrix(w, ldw, n, k, e));
    if (dx) MIC_TRY(check_matrix(dx, lddx, m, k, e));
    if (dw) MIC_TRY(check_matrix(dw, lddw, n, k, e));
    if (!aligned(dbias, e)) return MIC_STATUS_BAD_PARAM;
    if (need && (!workspace || !aligned(workspace, 16) || workspace_bytes < need)) return MIC_STATUS_BAD_PARAM;
    if (n == 0 && (!dx || k == 0)) return MIC_STATUS_SUCCESS;
    ProductType type;
    MIC_TRY(product_type(dtype, dtype, &type));
    const GradLayout g = grad_layout(handle->num_cu, type, m, n, k, false, true, even, slope || !even);
    uint8_t* ws = static_cast<uint8_t*>(workspace);
    // without an activation dz is dy, read where it is
    const bool own = slope && (dx || dw);
    if (n && (own || dbias)) {
        miconv::SlopeArgs s = {};
        s.rows = m, s.cols = n, s.act = act;
        s.dy = dy, s.lddy = lddy;
        s.pre = slope ? preact : nullptr, s.ldp = ldp;
        s.dz = own && m ? ws : nullptr, s.dz_pitch = g.pitch, s.up_at = g.pitch;
        s.sums = dbias ? reinterpret_cast<float*>(ws + g.dz) : nullptr;
        s.dbias = dbias;
        MIC_TRY(launched(miconv::launch_slope(device_type(dtype), s, handle->stream)));
    }
    return grad_products(handle, type, m, n, k, own ? ws : dy, own ? g.pitch : lddy, own ? g.pitch : n, 0, x, ldx, w, ldw, nullptr, 0,
                         dx, lddx, dw, lddw, nullptr, 0, ws + g.dz + g.sums, g.product);
}

mic_status mic_gated_linear_forward_workspace(mic_handle handle, mic_dtype dtype, int m, int n, int k, size_t* bytes)
{
    return forward_workspace(handle, Product::GATED, dtype, m, n, k, false, bytes);
}

mic_status mic_gated_linear_forward_workspace_aligned(mic_handle handle, mic_dtype dtype, int m, int n, int k, size_t* bytes)
{
    return forward_workspace(handle, Product::GATED, dtype, m, n, k, true, bytes);
}

mic_status mic_gated_linear_forward(mic_handle handle, mic_dtype dtype, mic_dtype out_dtype, mic_activation act,
                                    int fast_sums, int m, int n, int k, const void* x, int64_t ldx, const void* w_gate,
                                    int64_t ldg, const void* w_up, int64_t ldu, const float* x_scale,
                                    const float* w_gate_scale, const float* w_up_scale, void* y, int64_t ldy,
                                    void* gate, int64_t ldgate, void* up, int64_t ldup, void* workspace,
                                    size_t workspace_bytes)
{
    if (!handle) return MIC_STATUS_BAD_PARAM;
    ProductType type;
    MIC_TRY(product_type(dtype, out_dtype, &type, fast_sums != 0));
    if (!valid_act(act)) return MIC_STATUS_NOT_SUPPORTED;
    MIC_TRY(check_sizes(m, n, k));
    if (n >= kMaxSize / 2) return MIC_STATUS_NOT_SUPPORTED;
    if (m == 0 || n == 0) return MIC_STATUS_SUCCESS;
    const size_t e = size_of(dtype), o = size_of(out_dtype);
    MIC_TRY(check_matrix(x, ldx, m, k, e));
    MIC_TRY(check_matrix(w_gate, ldg, n, k, e));
    MIC_TRY(check_matrix(w_up, ldu, n, k, e));
    MIC_TRY(check_matrix(y, ldy, m, n, o));
    if ((gate == nullptr) != (up == nullptr)) return MIC_STATUS_BAD_PARAM;
    if (gate) {
        MIC_TRY(check_matrix(gate, ldgate, m, n, o));
        MIC_TRY(check_matrix(up, ldup, m, n, o));
    }
    const bool scaled = dtype == MIC_DTYPE_F8_E4M3;
    if (scaled != (x_scale != nullptr) || scaled != (w_gate_scale != nullptr) || scaled != (w_up_scale != nullptr))
        return MIC_STATUS_BAD_PARAM;
    if (!aligned(x_scale, 4) || !aligned(w_gate_scale, 4) || !aligned(w_up_scale, 4)) return MIC_STATUS_BAD_PARAM;
    ProductArgs p = {};
    p.a = static_cast<const uint8_t*>(x), p.lda = ldx * (int64_t)e;
    p.b = static_cast<const uint8_t*>(w_gate), p.ldb = ldg * (int64_t)e;
    p.b2 = static_cast<const uint8_t*>(w_up), p.ldb2 = ldu * (int64_t)e;
    p.M = m, p.N = n, p.K = k, p.k_segments = 1;
    p.act = act;
    p.y = y, p.ldy = ldy;
    p.x_scale = x_scale, p.w_scale = w_gate_scale, p.w2_scale = w_up_scale;
    p.pre = gate, p.ldp = ldgate;
    p.pre2 = up, p.ldp2 = ldup;
    return run_product(handle, Product::GATED, type, p, workspace, workspace_bytes);
}

mic_status mic_gated_linear_backward_workspace(mic_handle handle, mic_dtype dtype, int m, int n, int k,
                                               size_t* bytes)
{
    return backward_workspace(handle, dtype, m, n, k, true, false, true, bytes);
}

mic_status mic_gated_linear_backward_workspace_aligned(mic_handle handle, mic_dtype dtype, int m, int n, int k, size_t* bytes)
{
    return backward_workspace(handle, dtype, m, n, k, true, true, true, bytes);
}

mic_status mic_gated_linear_backward(mic_handle handle, mic_dtype dtype, mic_activation act, int m, int n, int k,
                                     const void* dy, int64_t lddy, const void* x, int64_t ldx, const void* w_gate,
                                     int64_t ldg, const void* w_up, int64_t ldu, const void* gate, int64_t ldgate,
                                     const void* up, int64_t ldup, void* dx, int64_t lddx, void* dw_gate,
                                     int64_t lddg, void* dw_up, int64_t lddu, void* workspace,
                                     size_t workspace_bytes)
{
    if (!handle) return MIC_STATUS_BAD_PARAM;
    const size_t e = size_of(dtype);
    const bool even = (!dw_gate || aligned_matrix(x, ldx * (int64_t)e))
                      && (!dx || (aligned_matrix(w_gate, ldg * (int64_t)e) && aligned_matrix(w_up, ldu * (int64_t)e) && ldg == ldu));
    size_t need;
    MIC_TRY(backward_workspace(handle, dtype, m, n, k, true, even, true, &need));
    if (!valid_act(act)) return MIC_STATUS_NOT_SUPPORTED;
    MIC_TRY(check_matrix(dy, lddy, m, n, e));
    MIC_TRY(check_matrix(gate, ldgate, m, n, e));
    MIC_TRY(check_matrix(up, ldup, m, n, e));
    if ((dw_gate == nullptr) != (dw_up == nullptr)) return MIC_STATUS_BAD_PARAM;
    if (dw_gate) {
        MIC_TRY(check_matrix(x, ldx, m, k, e));
        MIC_TRY(check_matrix(dw_gate, lddg, n, k, e));
        MIC_TRY(check_matrix(dw_up, lddu, n, k, e));
    }
    if (dx) {
        MIC_TRY(check_matrix(w_gate, ldg, n, k, e));
        MIC_TRY(check_matrix(w_up, ldu, n, k, e));
        MIC_TRY(check_matrix(dx, lddx, m, k, e));
    }
    if (need && (!workspace || !aligned(workspace, 16) || workspace_bytes < need)) return MIC_STATUS_BAD_PARAM;
    if ((!dx && !dw_gate) || k == 0) return MIC_STATUS_SUCCESS;
    ProductType type;
    MIC_TRY(product_type(dtype, dtype, &type));
    const GradLayout g = grad_layout(handle->num_cu, type, m, n, k, true, false, even, true);
    uint8_t* ws = static_cast<uint8_t*>(workspace);
    if (m && n) {
        miconv::SlopeArgs s = {};
        s.rows = m, s.cols = n, s.act = act;
        s.dy = dy, s.lddy = lddy;
        s.pre = gate, s.ldp = ldgate;
        s.up = up, s.ldu = ldup;
        s.dz = ws, s.dz_pitch = 2 * g.pitch, s.up_at = g.pitch;
        MIC_TRY(launched(miconv::launch_slope(device_type(dtype), s, handle->stream)));
    }
    // n == 0: dx is a sum of nothing, and the weights are never read
    const void* w2 = w_up ? w_up : ws;
    return grad_products(handle, type, m, n, k, ws, 2 * g.pitch, g.pitch, g.pitch, x, ldx, w_gate, ldg, w2, ldu, dx, lddx,
                         dw_gate, lddg, dw_up, lddu, ws + g.dz + g.sums, g.product);
}

}  // extern "C"
