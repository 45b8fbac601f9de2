// cross_entropy.cpp -- host side of the linear cross entropy: which way the logits go, in which pieces, and the calls
// put together from the products.
#include <stdio.h>

#include <cmath>

#include "product.h"

namespace {

using namespace miconv;

// Columns of a run of logits in memory: 1024, four a thread, where a row is long and rows are few; a row of 4096 is one
// run, finished where it is read.
constexpr int kRun = 1024, kWholeRow = 4096;
int run_of(int n) { return n <= kWholeRow ? kWholeRow : kRun; }
// What is held of the logits at one time: fp32 where a loss passes them through memory, dz in the tensors' type (and, where
// a gradient's pass through memory, fp32 logits for as many classes).  A piece is a product's columns: at 4096 rows of
// 4096 features 16384 of them keep every tile busy 8 rounds long.
constexpr int64_t kLogitsBytes = int64_t(1) << 28, kGradientBytes = int64_t(1) << 29;
constexpr int kPieceStep = 1024;                               // classes; also a piece of any number of rows has as many, each
                                                               // piece reading all of x: more than those bytes past 65536
                                                               // rows (a loss, fp32 gradients 131072, bf16 262144)
constexpr int kPieceMost = 1 << 19;                            // dz's rows stay short of 4 MB

// The share of all classes in fp32, below 1 there too: at 1 a target that a bias takes out would have 0 times infinity for a
// loss.
float share_of(double label_smoothing) { return std::min((float)label_smoothing, 0x1.fffffep-1f); }

ProductType type_of(mic_dtype d) { return d == MIC_DTYPE_F32 ? ProductType::F32 : ProductType::BF16; }
ProductType logits_type(ProductType t) { return t == ProductType::F32 ? ProductType::F32 : ProductType::BF16_F32; }

// Classes of a piece of m rows that takes at most `bytes`.
int piece_of(int64_t bytes, int m, int n, int element)
{
    const int64_t most = bytes / ((int64_t)m * element) / kPieceStep * kPieceStep;
    return (int)std::min<int64_t>({n, kPieceMost, std::max<int64_t>(most, kPieceStep)});
}

// Whether operands' rows, k long, can be read 16 bytes at a time.
struct Rows {
    bool x, w;
};
Rows rows_of(ProductType type, int k, bool x, bool w)
{
    const int64_t bytes = (int64_t)k * element_bytes(type);
    const bool even = bytes % 16 == 0 && bytes < kMaxPitchBytes / 2;
    return {x && even, w && even};
}

// Logits that pass through memory: the parts that their reduction is cut into, at the least.  Tiles of fp32 are slow, and a
// few more of them than the CUs are two rounds, the second all but empty; parts past what a product's own plan allows even
// the rounds out.  33184 classes, 260 tiles: of 3920 features 48 rows 273 -> 202 us, 128 rows 392 -> 323, of 2050
// features, whose rows whole tiles would copy, 48 rows 271 -> 124.  (Calls under a billion terms, some 30 us, are
// not worth the search.)
int logits_parts(int cus, ProductType type, int m, int n, int k, Rows rows)
{
    if (type != ProductType::F32 || (double)m * n * k < 1e9) return 1;
    int parts = 1;
    double us = 1e30;
    for (int s = 1; s <= 8 && s <= k / 128; ++s) {
        const Plan pl = plan_product(cus, Product::FORWARD, type, m, n, k, 1, rows.x, rows.w, s);
        if (pl.us < us) us = pl.us, parts = s;
    }
    return parts;
}
Plan plan_logits(int cus, ProductType type, int m, int n, int k, Rows rows)
{
    return plan_product(cus, Product::FORWARD, logits_type(type), m, n, k, 1, rows.x, rows.w, logits_parts(cus, type, m, n, k, rows));
}

// A product over aligned copies of operands that are not: the whole of x once, w a piece at a time.
struct Copies {
    int64_t pitch;                                             // bytes, 0: none
    size_t x, w;
    double us;
};
Copies copies_of(ProductType type, int m, int n, int piece, int k, Rows rows)
{
    Copies c = {};
    if (rows.x && rows.w) return c;
    c.pitch = align_up((int64_t)k * element_bytes(type), 16);
    if (!rows.x) c.x = (size_t)align_up(c.pitch * m, 256);
    if (!rows.w) c.w = (size_t)align_up(c.pitch * piece, 256);
    c.us = 2.0 * c.pitch * ((rows.x ? 0 : m) + (double)(rows.w ? 0 : n)) / kBytesPerUs + kLaunchUs;
    return c;
}

// An fp32 gradient's sum over thousands of terms is added up in parts: after the one term that is large, the target's, a
// single chain rounds every small one at the large one's size (dx over 50021 classes was 4.4e-6 off, the plain form 2.4e-6).
int gradient_parts(ProductType type, int terms) { return type == ProductType::F32 ? std::min((terms + 4095) / 4096, 256) : 1; }

// A product over all the classes of a piece ends in a round of tiles that leaves most CUs idle.  The classes after its
// whole rounds of 256 x 256 tiles are then a product of their own, on smaller tiles: the classes of the first, 0 for one
// product.  CLASS_GRAD's classes are its rows, the others' its columns.
Plan plan_classes(int cus, Product kind, ProductType type, int m, int n, int k)
{
    return kind == Product::CLASS_GRAD ? plan_product(cus, kind, type, n, k, m, 1, true, true, gradient_parts(type, m))
                                        : plan_product(cus, kind, type, m, n, k, 1, true, true);
}
int cut_of(int cus, Product kind, ProductType type, int m, int n, int k)
{
    if (type == ProductType::F32) return 0;
    const int64_t across = ((kind == Product::CLASS_GRAD ? k : m) + 255) / 256, rounds = across * ((n + 255) / 256) / cus;
    const int64_t first = rounds * cus / across * 256;
    if (first <= 0 || first >= n) return 0;
    const Plan whole = plan_classes(cus, kind, type, m, n, k), a = plan_classes(cus, kind, type, m, (int)first, k),
               b = plan_classes(cus, kind, type, m, n - (int)first, k);
    if (!planned(whole) || !planned(a) || !planned(b) || a.splits > 1) return 0;
    return a.us + b.us + kLaunchUs < whole.us ? (int)first : 0;
}

// f(first class, classes) for one product or two.
template <class F> mic_status in_cuts(int n, int cut, F f)
{
    MIC_TRY(f(0, cut ? cut : n));
    return cut ? f(cut, n - cut) : MIC_STATUS_SUCCESS;
}

// How a call goes.
struct Way {
    bool fused;              // the logits stay in the tiles that make them
    int piece;               // classes at a time
    Plan plan;               // of the (first) piece's logits
    Copies copies;
    int runs;                // forward: partial results a row
    size_t copy_bytes, logits, product, total;
    // gradient
    size_t dz, sums, sum;
    int64_t dz_pitch, ld_logits;
};

// Bytes of a product over the pieces' two sizes.
template <class Bytes> size_t over_pieces(int n, int piece, Bytes bytes)
{
    const size_t whole = bytes(piece);
    return n % piece ? std::max(whole, bytes(n % piece)) : whole;
}

// Runs that a fused product over `classes` leaves.
int runs_of(const Plan& pl, int classes)
{
    const int columns = pl.few ? 8 : loss_columns(pl.fast_tile);
    return (classes + columns - 1) / columns;
}

// A fused forward product's cut, and the plan of one of its parts.
int loss_cut(int cus, const Way& w, ProductType type, int m, int n, int k)
{
    return w.plan.few ? 0 : cut_of(cus, Product::LOSS, type, m, n, k);
}
Plan loss_plan(int cus, const Way& w, ProductType type, int m, int n, int classes, int k)
{
    return classes == n ? w.plan : plan_product(cus, Product::LOSS, type, m, classes, k, 1, true, true);
}

Way forward_way(int cus, ProductType type, int m, int n, int k, Rows rows)
{
    Way fused = {}, memory = {};
    // few rows as they lie, whole tiles from aligned rows, copied first where they are not
    fused.fused = true;
    fused.piece = n;
    fused.copies = copies_of(type, m, n, n, k, rows);
    fused.plan = plan_product(cus, Product::LOSS, type, m, n, k, 1, true, true);
    const Plan few = plan_product(cus, Product::LOSS, type, m, n, k, 1, rows.x && rows.w, rows.x && rows.w);
    if (few.few && few.us <= fused.plan.us + fused.copies.us) fused.plan = few, fused.copies = {};
    memory.piece = piece_of(kLogitsBytes, m, n, 4);
    memory.plan = plan_logits(cus, type, m, memory.piece, k, rows);
    const double pieces = (n + memory.piece - 1) / memory.piece;
    const double fused_us = fused.plan.us + fused.copies.us + 2.0 * m * ((n + 63) / 64) * 8 / kBytesPerUs;
    const double memory_us = pieces * (memory.plan.us + kLaunchUs) + 2.0 * m * (double)n * 4 / kBytesPerUs;
    Way w = planned(fused.plan) && fused_us < memory_us ? fused : memory;
    if (w.fused) {
        w.runs = 0;
        in_cuts(n, loss_cut(cus, w, type, m, n, k), [&](int first, int classes) {
            w.runs += runs_of(loss_plan(cus, w, type, m, n, classes, k), classes);
            return MIC_STATUS_SUCCESS;
        });
        w.copy_bytes = w.copies.x + w.copies.w;
    } else {
        w.runs = 0;
        for (int v = 0; v < n; v += w.piece) w.runs += (std::min(w.piece, n - v) + run_of(n) - 1) / run_of(n);
        w.ld_logits = align_up(w.piece, 4);
        w.logits = (size_t)align_up((int64_t)m * w.ld_logits * 4, 256);
        w.product = over_pieces(n, w.piece, [&](int columns) {
            return plan_logits(cus, type, m, columns, k, rows).bytes;
        });
        w.product = (size_t)align_up(w.product, 256);
    }
    // the runs' statistics, the targets' logits and the rows' losses
    w.total = w.copy_bytes + w.logits + w.product + (size_t)align_up((int64_t)m * (12 * (int64_t)w.runs + 8), 256);
    return w;
}

// Sums of each column that a fused product over `classes` leaves.
int sum_groups(int cus, ProductType type, int m, int classes, int k)
{
    const int rows = loss_rows(plan_product(cus, Product::LOGITS_GRAD, type, m, classes, k, 1, true, true).fast_tile);
    return (m + rows - 1) / rows;
}

int weight_cut(int cus, const Way& w, ProductType type, int m, int columns, int k)
{
    return w.fused ? cut_of(cus, Product::CLASS_GRAD, type, m, columns, k) : 0;
}

Way backward_way(int cus, ProductType type, int m, int n, int k, Rows rows, bool bias)
{
    const int e = element_bytes(type);
    Way fused = {}, memory = {};
    fused.fused = true;
    fused.piece = memory.piece = piece_of(kGradientBytes, m, n, e);
    fused.copies = copies_of(type, m, n, fused.piece, k, rows);
    fused.plan = plan_product(cus, Product::LOGITS_GRAD, type, m, fused.piece, k, 1, true, true);
    memory.plan = plan_logits(cus, type, m, memory.piece, k, rows);
    const double pieces = (n + fused.piece - 1) / fused.piece;
    const double fused_us = pieces * (fused.plan.us + (bias ? kLaunchUs : 0.0)) + fused.copies.us;
    const double memory_us = pieces * (memory.plan.us + kLaunchUs) + (double)m * n * (8 + e) / kBytesPerUs;
    Way w = planned(fused.plan) && fused_us < memory_us ? fused : memory;
    const Rows now = w.fused ? Rows{true, true} : rows;
    w.copy_bytes = w.copies.x + w.copies.w;
    w.dz_pitch = align_up(w.piece, 64);
    w.dz = (size_t)align_up((int64_t)m * w.dz_pitch * e, 256);
    if (bias)
        w.sums = over_pieces(n, w.piece, [&](int columns) {
            size_t most = (size_t)slope_row_groups(m, columns) * columns;
            if (w.fused) {
                most = 0;
                in_cuts(columns, cut_of(cus, Product::LOGITS_GRAD, type, m, columns, k), [&](int, int classes) {
                    most = std::max(most, (size_t)sum_groups(cus, type, m, classes, k) * classes);
                    return MIC_STATUS_SUCCESS;
                });
            }
            return (size_t)align_up(most * 4, 256);
        });
    if (w.piece < n) w.sum = (size_t)align_up((int64_t)m * align_up(k, 8) * 4, 256);
    if (!w.fused) {
        w.ld_logits = align_up(w.piece, 4);
        w.logits = (size_t)align_up((int64_t)m * w.ld_logits * 4, 256);
    }
    w.product = over_pieces(n, w.piece, [&](int columns) {
        size_t most = plan_product(cus, Product::INPUT_SUM, type, m, k, columns, 1, true, now.w, gradient_parts(type, columns)).bytes;
        in_cuts(columns, weight_cut(cus, w, type, m, columns, k), [&](int, int classes) {
            most = std::max(most, plan_product(cus, Product::CLASS_GRAD, type, classes, k, m, 1, true, now.x, gradient_parts(type, m)).bytes);
            return MIC_STATUS_SUCCESS;
        });
        if (!w.fused)
            most = std::max(most, plan_logits(cus, type, m, columns, k, rows).bytes);
        return most;
    });
    w.product = (size_t)align_up(w.product, 256);
    w.total = w.copy_bytes + w.dz + w.sums + w.sum + w.logits + w.product;
    return w;
}

// Whether dx and dw go side by side: two small products, one after the other, each leave CUs idle and wait out memory's
// latency alone (952 x 1152 of 704 features: 12.4 and 11.7 us, together 14.2).  Aligned operands, whole products on
// 128 x 128 tiles, no more of them than the CUs hold at once.
bool pairs(int cus, const Way& w, ProductType type, int m, int n, int k, Rows rows)
{
    if (w.piece < n || !(w.fused || (rows.x && rows.w))) return false;
    if (w.fused && cut_of(cus, Product::CLASS_GRAD, type, m, n, k)) return false;
    auto small = [](const Plan& pl) { return pl.fast && pl.fast_tile == FastTile::T128x128 && pl.splits == 1 && !pl.pack_a && !pl.pack_b; };
    if (!small(plan_product(cus, Product::INPUT_SUM, type, m, k, n, 1, true, true, gradient_parts(type, n)))
        || !small(plan_product(cus, Product::CLASS_GRAD, type, n, k, m, 1, true, true, gradient_parts(type, m))))
        return false;
    const int64_t across = (k + 127) / 128;
    return ((m + 127) / 128 + (n + 127) / 128) * across <= 2 * cus;
}

mic_status check_loss(mic_dtype dtype, int m, int n, int k)
{
    MIC_TRY(check_sizes(m, n, k));
    return plain_type(dtype) ? MIC_STATUS_SUCCESS : MIC_STATUS_NOT_SUPPORTED;
}

// The most a call of these sizes takes, whatever its rows' alignment; or aligned ones.
template <class Bytes> size_t most_rows(ProductType type, int k, bool aligned, Bytes bytes)
{
    if (aligned) return bytes(rows_of(type, k, true, true));
    size_t most = 0;
    for (int a = 0; a < 4; ++a) most = std::max(most, bytes(rows_of(type, k, a & 1, a & 2)));
    return most;
}

mic_status loss_workspace(mic_handle h, mic_dtype dtype, int m, int n, int k, bool backward, bool aligned, size_t* bytes)
{
    if (!bytes) return MIC_STATUS_BAD_PARAM;
    MIC_TRY(check_loss(dtype, m, n, k));
    *bytes = 0;
    if (!m || !n) return MIC_STATUS_SUCCESS;
    const ProductType type = type_of(dtype);
    *bytes = most_bytes(h, [&](int cus) {
        return most_rows(type, k, aligned, [&](Rows rows) {
            return backward ? backward_way(cus, type, m, n, k, rows, true).total : forward_way(cus, type, m, n, k, rows).total;
        });
    });
    return MIC_STATUS_SUCCESS;
}

mic_status loss_name(mic_handle h, mic_dtype dtype, int m, int n, int k, bool backward, int aligned, char* buf, size_t buflen)
{
    MIC_TRY(check_loss(dtype, m, n, k));
    if (!m || !n) return give_name("nothing", buf, buflen);
    const ProductType type = type_of(dtype);
    const Rows rows = rows_of(type, k, aligned != 0, aligned != 0);
    const Way w = backward ? backward_way(cus_of(h), type, m, n, k, rows, true) : forward_way(cus_of(h), type, m, n, k, rows);
    if (!planned(w.plan)) return MIC_STATUS_NOT_SUPPORTED;
    char text[192], product[64];
    if (w.fused) {
        const Product kind = backward ? Product::LOGITS_GRAD : Product::LOSS;
        int at = snprintf(text, sizeof(text), "fused");
        const int cut = backward ? cut_of(cus_of(h), kind, type, m, w.piece, k) : loss_cut(cus_of(h), w, type, m, n, k);
        in_cuts(w.piece, cut, [&](int first, int classes) {
            describe(classes == w.piece ? w.plan : plan_product(cus_of(h), kind, type, m, classes, k, 1, true, true), product,
                     sizeof(product));
            at += snprintf(text + at, sizeof(text) - at, "%s %s", first ? " +" : "", product);
            return MIC_STATUS_SUCCESS;
        });
        snprintf(text + at, sizeof(text) - at, "%s, %d pieces", w.copies.pitch ? " copies" : "", (n + w.piece - 1) / w.piece);
    } else {
        describe(w.plan, product, sizeof(product));
        snprintf(text, sizeof(text), "%s, %d pieces", product, (n + w.piece - 1) / w.piece);
    }
    return give_name(text, buf, buflen);
}

// The operands of a product on x and w: where they lie, or aligned copies of them.
struct Operands {
    const uint8_t *x, *w;
    int64_t ldx, ldw;        // bytes
    int columns;             // elements of a row, zeros past k
};

mic_status copy_rows(mic_handle h, const Copies& c, int64_t row_bytes, bool with_x, int m, int columns, Operands& o, uint8_t*& at)
{
    PackJob jobs[2];
    int count = 0;
    if (with_x && c.x) jobs[count++] = {o.x, o.ldx, m, row_bytes, at, c.pitch};
    if (c.w) jobs[count++] = {o.w, o.ldw, columns, row_bytes, at + c.x, c.pitch};
    return count ? launched(launch_pack(jobs, count, h->stream)) : MIC_STATUS_SUCCESS;
}

}  // namespace

extern "C" {

mic_status mic_linear_cross_entropy_workspace(mic_handle handle, mic_dtype dtype, int m, int n, int k, size_t* bytes)
{
    return loss_workspace(handle, dtype, m, n, k, false, false, bytes);
}

mic_status mic_linear_cross_entropy_workspace_aligned(mic_handle handle, mic_dtype dtype, int m, int n, int k, size_t* bytes)
{
    return loss_workspace(handle, dtype, m, n, k, false, true, bytes);
}

mic_status mic_linear_cross_entropy(mic_handle handle, mic_dtype dtype, mic_reduction reduction, int m, int n, int k,
                                    const void* x, int64_t ldx, const void* w, int64_t ldw, const void* bias,
                                    const int64_t* target, int64_t ignore_index, double label_smoothing, float* loss,
                                    float* lse, float* count, void* workspace, size_t workspace_bytes)
{
    if (!handle) return MIC_STATUS_BAD_PARAM;
    MIC_TRY(check_loss(dtype, m, n, k));
    if ((int)reduction < 0 || (int)reduction > (int)MIC_REDUCTION_MEAN) return MIC_STATUS_NOT_SUPPORTED;
    if (!(label_smoothing >= 0.0 && label_smoothing < 1.0)) return MIC_STATUS_BAD_PARAM;
    const bool each = reduction == MIC_REDUCTION_NONE;
    if (m == 0 && each) return MIC_STATUS_SUCCESS;
    if (n == 0) return MIC_STATUS_BAD_PARAM;                   // a distribution over nothing
    const size_t e = size_of(dtype);
    MIC_TRY(check_matrix(x, ldx, m, k, e));
    MIC_TRY(check_matrix(w, ldw, m ? n : 0, k, e));
    if (!loss || !aligned(loss, 4) || !aligned(bias, e)) return MIC_STATUS_BAD_PARAM;
    if (m && (!lse || !aligned(lse, 4) || !target || !aligned(target, 8))) return MIC_STATUS_BAD_PARAM;
    if (!each && (!count || !aligned(count, 4))) return MIC_STATUS_BAD_PARAM;
    LossArgs a = {};
    a.target = target, a.ignore = ignore_index, a.classes = n, a.smooth = share_of(label_smoothing);
    if (m == 0) return launched(launch_loss_reduce(a, 0, loss, reduction == MIC_REDUCTION_MEAN, loss, count, handle->stream));

    const ProductType type = type_of(dtype);
    const Rows rows = rows_of(type, k, aligned_matrix(x, ldx * (int64_t)e), aligned_matrix(w, ldw * (int64_t)e));
    const Way way = forward_way(handle->num_cu, type, m, n, k, rows);
    if (!planned(way.plan)) return MIC_STATUS_NOT_SUPPORTED;
    if (!workspace || !aligned(workspace, 16) || workspace_bytes < way.total) return MIC_STATUS_BAD_PARAM;
    uint8_t* ws = static_cast<uint8_t*>(workspace);
    uint8_t* copies = ws;
    uint8_t* logits = copies + way.copy_bytes;
    uint8_t* space = logits + way.logits;
    a.part = reinterpret_cast<float*>(space + way.product);
    a.part_z = label_smoothing > 0.0 ? a.part + 2 * (int64_t)way.runs * m : nullptr;
    a.hit = a.part + 3 * (int64_t)way.runs * m;
    float* row_loss = each ? loss : a.hit + m;
    Operands o = {static_cast<const uint8_t*>(x), static_cast<const uint8_t*>(w), ldx * (int64_t)e, ldw * (int64_t)e, k};
    if (way.copies.pitch) {
        MIC_TRY(copy_rows(handle, way.copies, (int64_t)k * e, true, m, n, o, copies));
        if (way.copies.x) o.x = copies, o.ldx = way.copies.pitch;
        if (way.copies.w) o.w = copies + way.copies.x, o.ldw = way.copies.pitch;
        o.columns = (int)(way.copies.pitch / (int64_t)e);
    }
    auto product = [&](int first, int columns) {
        LossProductArgs p = {};
        p.cus = handle->num_cu;
        p.a = o.x, p.lda = o.ldx;
        p.b = o.w + (int64_t)first * o.ldw, p.ldb = o.ldw;
        p.M = m, p.N = columns, p.K = k, p.k_segments = 1, p.a_K = o.columns;
        return p;
    };
    auto bias_at = [&](int first) { return bias ? static_cast<const uint8_t*>(bias) + (int64_t)first * e : nullptr; };
    int run = 0;
    if (way.fused) {
        MIC_TRY(in_cuts(n, loss_cut(handle->num_cu, way, type, m, n, k), [&](int first, int columns) {
            LossProductArgs p = product(first, columns);
            p.loss = a;
            p.loss.first = first, p.loss.part_first = run;
            p.bias = bias_at(first);
            run += runs_of(loss_plan(handle->num_cu, way, type, m, n, columns, k), columns);
            return run_product(handle, Product::LOSS, type, p, nullptr, 0);
        }));
    } else {
        for (int v = 0; v < n; v += way.piece) {
            const int columns = std::min(way.piece, n - v);
            LossProductArgs p = product(v, columns);
            p.y = logits, p.ldy = way.ld_logits;
            Sums sums;
            p.splits = logits_parts(handle->num_cu, type, m, columns, k, rows);
            MIC_TRY(run_product(handle, Product::FORWARD, logits_type(type), p, space, way.product, &sums));
            LossRowsArgs r = {};
            r.loss = a;
            r.loss.first = v, r.loss.part_first = run;
            r.rows = m, r.cols = columns;
            r.z = sums.data, r.ld = sums.ld, r.splits = sums.splits;
            r.bias = bias_at(v);
            r.run = run_of(n);
            if (way.runs == 1) r.lse = lse, r.row_loss = row_loss;
            MIC_TRY(launched(launch_loss_rows(device_type(dtype), r, handle->stream)));
            run += (columns + r.run - 1) / r.run;
        }
    }
    if (way.fused || way.runs > 1) MIC_TRY(launched(launch_loss_join(a, m, way.runs, lse, row_loss, handle->stream)));
    if (each) return MIC_STATUS_SUCCESS;
    return launched(launch_loss_reduce(a, m, row_loss, reduction == MIC_REDUCTION_MEAN, loss, count, handle->stream));
}

mic_status mic_linear_cross_entropy_kernel_name(mic_handle handle, mic_dtype dtype, int m, int n, int k, int aligned, char* buf,
                                                size_t buflen)
{
    return loss_name(handle, dtype, m, n, k, false, aligned, buf, buflen);
}

mic_status mic_linear_cross_entropy_backward_workspace(mic_handle handle, mic_dtype dtype, int m, int n, int k, size_t* bytes)
{
    return loss_workspace(handle, dtype, m, n, k, true, false, bytes);
}

mic_status mic_linear_cross_entropy_backward_workspace_aligned(mic_handle handle, mic_dtype dtype, int m, int n, int k,
                                                               size_t* bytes)
{
    return loss_workspace(handle, dtype, m, n, k, true, true, bytes);
}

mic_status mic_linear_cross_entropy_backward(mic_handle handle, mic_dtype dtype, int m, int n, int k, const float* dloss,
                                             int dloss_rows, const void* x, int64_t ldx, const void* w, int64_t ldw,
                                             const void* bias, const int64_t* target, int64_t ignore_index,
                                             double label_smoothing, const float* lse, const float* count, void* dx,
                                             int64_t lddx, void* dw, int64_t lddw, void* dbias, void* workspace,
                                             size_t workspace_bytes)
{
    if (!handle) return MIC_STATUS_BAD_PARAM;
    MIC_TRY(check_loss(dtype, m, n, k));
    if (!(label_smoothing >= 0.0 && label_smoothing < 1.0)) return MIC_STATUS_BAD_PARAM;
    const size_t e = size_of(dtype);
    MIC_TRY(check_matrix(x, ldx, m, k, e));
    MIC_TRY(check_matrix(w, ldw, m ? n : 0, k, e));
    if (dx) MIC_TRY(check_matrix(dx, lddx, m, k, e));
    if (dw) MIC_TRY(check_matrix(dw, lddw, n, k, e));
    if (!aligned(bias, e) || !aligned(dbias, e) || !aligned(count, 4)) return MIC_STATUS_BAD_PARAM;
    if (m && (!dloss || !aligned(dloss, 4) || !lse || !aligned(lse, 4) || !target || !aligned(target, 8)))
        return MIC_STATUS_BAD_PARAM;
    if (n == 0) return m ? MIC_STATUS_BAD_PARAM : MIC_STATUS_SUCCESS;
    if (!dx && !dw && !dbias) return MIC_STATUS_SUCCESS;
    if (m == 0) {
        // no rows: the weights' gradients are sums of nothing
        if (dw && k) {
            ProductArgs p = {};
            p.M = n, p.N = k, p.K = 0, p.k_segments = 1;
            p.m_pitch = INT32_MAX, p.m_valid = n;
            p.y = dw, p.ldy = lddw;
            MIC_TRY(run_product(handle, Product::WEIGHT_GRAD, type_of(dtype), p, nullptr, 0));
        }
        return dbias ? launched(launch_column_join(device_type(dtype), nullptr, 0, n, dbias, handle->stream)) : MIC_STATUS_SUCCESS;
    }
    const ProductType type = type_of(dtype);
    const Rows rows = rows_of(type, k, aligned_matrix(x, ldx * (int64_t)e), aligned_matrix(w, ldw * (int64_t)e));
    const Way way = backward_way(handle->num_cu, type, m, n, k, rows, true);
    if (!planned(way.plan)) return MIC_STATUS_NOT_SUPPORTED;
    if (!workspace || !aligned(workspace, 16) || workspace_bytes < way.total) return MIC_STATUS_BAD_PARAM;
    uint8_t* copies = static_cast<uint8_t*>(workspace);
    uint8_t* dz = copies + way.copy_bytes;
    float* column_sums = reinterpret_cast<float*>(dz + way.dz);
    float* sum = reinterpret_cast<float*>(dz + way.dz + way.sums);
    uint8_t* logits = dz + way.dz + way.sums + way.sum;
    uint8_t* space = logits + way.logits;
    LossArgs a = {};
    a.target = target, a.ignore = ignore_index, a.classes = n, a.smooth = share_of(label_smoothing);
    a.lse = lse, a.dloss = dloss, a.dloss_rows = dloss_rows, a.count = count;
    for (int v = 0; v < n; v += way.piece) {
        const int columns = std::min(way.piece, n - v);
        const int64_t pitch = align_up(columns, 64);
        Operands o = {static_cast<const uint8_t*>(x), static_cast<const uint8_t*>(w) + (int64_t)v * ldw * (int64_t)e,
                      ldx * (int64_t)e, ldw * (int64_t)e, k};
        if (way.copies.pitch) {
            MIC_TRY(copy_rows(handle, way.copies, (int64_t)k * e, v == 0, m, columns, o, copies));
            if (way.copies.x) o.x = copies, o.ldx = way.copies.pitch;
            if (way.copies.w) o.w = copies + way.copies.x, o.ldw = way.copies.pitch;
            o.columns = (int)(way.copies.pitch / (int64_t)e);
        }
        auto product = [&](int first, int classes) {
            LossProductArgs p = {};
            p.cus = handle->num_cu;
            p.a = o.x, p.lda = o.ldx;
            p.b = o.w + (int64_t)first * o.ldw, p.ldb = o.ldw;
            p.M = m, p.N = classes, p.K = k, p.k_segments = 1, p.a_K = o.columns;
            p.bias = bias ? static_cast<const uint8_t*>(bias) + (int64_t)(v + first) * e : nullptr;
            return p;
        };
        void* piece_dbias = dbias ? static_cast<uint8_t*>(dbias) + (int64_t)v * e : nullptr;
        if (way.fused) {
            MIC_TRY(in_cuts(columns, cut_of(handle->num_cu, Product::LOGITS_GRAD, type, m, columns, k), [&](int first, int classes) {
                LossProductArgs p = product(first, classes);
                p.loss = a;
                p.loss.first = v + first;
                // the last classes' product also clears what pads dz's rows
                p.y = dz + first * (int64_t)e, p.ldy = pitch, p.y_columns = first + classes == columns ? (int)pitch - first : classes;
                p.sums = dbias ? column_sums : nullptr;
                MIC_TRY(run_product(handle, Product::LOGITS_GRAD, type, p, nullptr, 0));
                if (!dbias) return MIC_STATUS_SUCCESS;
                return launched(launch_column_join(device_type(dtype), column_sums,
                                                   sum_groups(handle->num_cu, type, m, classes, k), classes,
                                                   static_cast<uint8_t*>(piece_dbias) + first * (int64_t)e, handle->stream));
            }));
        } else {
            LossProductArgs p = product(0, columns);
            LossRowsArgs r = {};
            r.bias = p.bias;
            p.bias = nullptr;
            p.y = logits, p.ldy = way.ld_logits;
            Sums sums;
            p.splits = logits_parts(handle->num_cu, type, m, columns, k, rows);
            MIC_TRY(run_product(handle, Product::FORWARD, logits_type(type), p, space, way.product, &sums));
            r.loss = a;
            r.loss.first = v;
            r.rows = m, r.cols = columns;
            r.z = sums.data, r.ld = sums.ld, r.splits = sums.splits;
            r.dz = dz, r.dz_pitch = pitch;
            r.sums = dbias ? column_sums : nullptr, r.dbias = piece_dbias;
            MIC_TRY(launched(launch_loss_gradient(device_type(dtype), r, handle->stream)));
        }
        auto input = [&] {
            LossProductArgs g = {};
            g.cus = handle->num_cu;
            g.a = dz, g.lda = pitch * (int64_t)e;
            g.b = o.w, g.ldb = o.ldw;
            g.M = m, g.N = k, g.K = columns, g.a_K = (int)pitch, g.b_rows = o.columns;
            g.k_segments = 1;
            g.y = dx, g.ldy = lddx;
            g.splits = gradient_parts(type, columns);
            g.loss = a;
            g.sum = sum, g.ld_sum = align_up(k, 8), g.sum_first = v == 0, g.sum_last = v + columns == n;
            return g;
        };
        auto weights = [&](int first, int classes) {
            LossProductArgs g = {};
            g.cus = handle->num_cu;
            g.a = dz + first * (int64_t)e, g.lda = pitch * (int64_t)e;
            g.b = o.x, g.ldb = o.ldx;
            g.M = classes, g.N = k, g.K = m, g.b_rows = o.columns;
            g.a_rows = first + classes == columns ? (int)pitch - first : classes;
            g.k_segments = 1;
            g.y = static_cast<uint8_t*>(dw) + (int64_t)(v + first) * lddw * (int64_t)e, g.ldy = lddw;
            g.splits = gradient_parts(type, m);
            g.loss = a;
            g.sum_first = g.sum_last = true;
            return g;
        };
        if (dx && dw && k && pairs(handle->num_cu, way, type, m, n, k, rows)) {
            LossProductArgs first = input(), second = weights(0, columns);
            MIC_TRY(run_pair(handle, type, first, second));
            continue;
        }
        if (dx && k) {
            LossProductArgs g = input();
            MIC_TRY(run_product(handle, Product::INPUT_SUM, type, g, space, way.product));
        }
        if (dw && k)
            MIC_TRY(in_cuts(columns, weight_cut(handle->num_cu, way, type, m, columns, k), [&](int first, int classes) {
                LossProductArgs g = weights(first, classes);
                return run_product(handle, Product::CLASS_GRAD, type, g, space, way.product);
            }));
    }
    return MIC_STATUS_SUCCESS;
}

mic_status mic_linear_cross_entropy_backward_kernel_name(mic_handle handle, mic_dtype dtype, int m, int n, int k, int aligned,
                                                         char* buf, size_t buflen)
{
    return loss_name(handle, dtype, m, n, k, true, aligned, buf, buflen);
}

}  // extern "C"
