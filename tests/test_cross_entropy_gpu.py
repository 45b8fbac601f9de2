"""GPU parity of the linear cross entropy and its gradients against plain 64-bit forms (bounds in training_ref)."""
import pytest
import torch

import convolution_forward_conv2d_amd as mic
import training_ref as T

pytestmark = pytest.mark.gpu

F32, BF16 = torch.float32, torch.bfloat16
DEV = "cuda:0"


def values(seed, *shape, std=1.0, dtype=F32):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(shape, generator=g) * std).to(dtype).to(DEV)


def classes(seed, m, n, ignored=0):
    g = torch.Generator().manual_seed(seed)
    t = torch.randint(0, n, (m,), generator=g)
    t[0], t[-1] = 0, n - 1
    if ignored:
        t[::ignored] = -100
    return t.to(DEV)


def run(x, w, bias, target, reduction, a=0.0, **kw):
    """Forward and gradients, checked."""
    got = mic.linear_cross_entropy(x, w, target, bias=bias, reduction=reduction, label_smoothing=a, **kw)
    want = T.cross_entropy(x, w, bias, target, reduction, a=a, ignore=kw.get("ignore_index", -100))
    assert got.loss.dtype is F32 and got.loss.shape == (target.shape if reduction == "none" else ())
    T.check(got.lse, want["lse"], "lse")
    T.check(got.loss, want["loss"], "loss")
    ignore = kw.get("ignore_index", -100)
    if reduction == "none":
        assert got.count is None
        dloss = values(9, target.numel())
    else:
        assert float(got.count) == float((target != ignore).sum())
        dloss = torch.tensor(1.25, device=DEV)
    count = got.count if reduction == "mean" else None
    grads = mic.linear_cross_entropy_backward(dloss, x, w, target, got.lse, bias=bias, count=count, label_smoothing=a, **kw)
    ref = T.cross_entropy_backward(dloss, x, w, bias, target, got.lse, count, ignore=ignore, a=a)
    for g, r, name in zip(grads, ref, ("dx", "dw", "dbias")):
        if name == "dbias" and bias is None:
            assert g is None
            continue
        assert g.dtype is x.dtype
        T.check(g, r, name)
    return got, grads


# one row, one class, one feature; few rows; one past and short of tiles; odd everything; several runs of 4096 classes
SIZES = [(1, 1, 1), (1, 5, 8), (2, 1000, 64), (1, 9001, 40), (3, 33, 31), (7, 4096, 136), (16, 4097, 512), (31, 65, 257),
         (33, 127, 129), (64, 64, 64), (65, 63, 65), (100, 72, 1000), (128, 1000, 512), (129, 1001, 63), (257, 129, 520),
         (300, 2049, 96), (513, 1531, 192), (640, 5003, 264), (1024, 3000, 128), (1100, 2304, 129)]


@pytest.mark.parametrize("m,n,k", SIZES)
@pytest.mark.parametrize("dtype", [F32, BF16])
def test_sizes(m, n, k, dtype):
    x, w, b = values(1, m, k, dtype=dtype), values(2, n, k, std=2 * k ** -0.5, dtype=dtype), values(3, n, dtype=dtype)
    run(x, w, None, classes(4, m, n), "mean")
    run(x, w, b, classes(5, m, n, ignored=3 if m > 3 else 0), "none", a=0.1)
    run(x, w, b, classes(6, m, n, ignored=2 if m > 2 else 0), "sum", ignore_index=-100)


# sizes that reach each way of the logits: every tile they stay in, both ways through memory, split sums, copies of
# unaligned rows (the name holds for aligned operands where k allows)
WAYS = [("fused fast 256x256, 1", BF16, 1500, 8200, 64), ("fused fast 256x192, 1", BF16, 1000, 8200, 64),
        ("fused fast 192x256, 1", BF16, 515, 20011, 40), ("fused fast 256x128, 1", BF16, 129, 20011, 40),
        ("fused fast 128x256, 1", BF16, 770, 8200, 64), ("fused fast 128x128, 1", BF16, 260, 135, 256),
        ("fused fast 256x256 + fast 128x128, 1", BF16, 1024, 17003, 1024),
        ("fused fast 128x128, 1", F32, 200, 8200, 64), ("fused fast 128x64, 1", F32, 70, 130, 64),
        ("fused fast 64x128, 1", F32, 129, 8200, 64), ("fused fast 128x128 copies", BF16, 1000, 2000, 71),
        ("fused fast 128x64 copies", F32, 1000, 1001, 65), ("any 64x64 split 4", BF16, 33, 130, 1001), ("any 64x64", BF16, 33, 130, 33),
        ("any 128x128 split 8", BF16, 200, 2500, 2047), ("fast 128x64 split 8 pack a pack b", F32, 33, 130, 1001),
        ("fast 128x128 split 4", BF16, 260, 130, 1024), ("fast 64x128 split 8", F32, 64, 2500, 1024), ("fused few", BF16, 2, 300, 100), ("fused few", BF16, 11, 3001, 100),
        ("fused few", F32, 20, 300, 100), ("fused few", F32, 1, 9001, 33),
        ("few", BF16, 16, 517, 2000), ("few", F32, 2, 700, 40)]


@pytest.mark.parametrize("way,dtype,m,n,k", WAYS)
def test_every_way(way, dtype, m, n, k):
    code = mic.MIC_DTYPE_BF16 if dtype is BF16 else mic.MIC_DTYPE_F32
    names = [f(mic.handle_for(), code, m, n, k) for f in (mic.mic_linear_cross_entropy_kernel_name,
                                                          mic.mic_linear_cross_entropy_backward_kernel_name)]
    assert any(name.startswith(way) for name in names), names
    x, w, b = values(1, m, k, dtype=dtype), values(2, n, k, std=2 * k ** -0.5, dtype=dtype), values(3, n, dtype=dtype)
    run(x, w, b, classes(4, m, n, ignored=5 if m > 5 else 0), "mean", a=0.2)
    run(x, w, None, classes(4, m, n), "none")


@pytest.mark.parametrize("way,m,n,k", [("fused fast 64x128", 40, 33184, 1024), ("split", 40, 33184, 2048), ("split", 47, 33000, 1025),
                                       ("fused fast 64x128", 130, 33184, 1000), ("fused fast 64x128", 130, 33184, 2100),
                                       ("split", 128, 33184, 3920)])
def test_parts_past_a_round(way, m, n, k):
    """Few more fp32 tiles than CUs: the reduction in parts, more of them than fill the CUs twice."""
    name = mic.mic_linear_cross_entropy_kernel_name(mic.handle_for(), mic.MIC_DTYPE_F32, m, n, k)
    assert way in name, name
    x, w, b = values(1, m, k), values(2, n, k, std=2 * k ** -0.5), values(3, n)
    run(x, w, b, classes(4, m, n, ignored=5), "mean", a=0.2)


@pytest.mark.parametrize("m,n,k", [(1000, 9000, 64), (2049, 4099, 72)])
@pytest.mark.parametrize("dtype", [F32, BF16])
def test_larger(m, n, k, dtype):
    x, w, b = values(1, m, k, dtype=dtype), values(2, n, k, std=2 * k ** -0.5, dtype=dtype), values(3, n, dtype=dtype)
    run(x, w, b, classes(4, m, n, ignored=7), "mean", a=0.1)
    run(x, w, None, classes(4, m, n, ignored=7), "mean")


@pytest.mark.parametrize("dtype,m,n,k,backward", [(F32, 4096, 33000, 8, "2 pieces"), (BF16, 8192, 33000, 16, "2 pieces"),
                                                  (F32, 4096, 70000, 9, "3 pieces"), (BF16, 3, 530000, 8, "2 pieces")])
def test_pieces(dtype, m, n, k, backward):
    """More gradients than are held at a time: dx adds up over pieces, the last one smaller."""
    code = mic.MIC_DTYPE_BF16 if dtype is BF16 else mic.MIC_DTYPE_F32
    assert backward in mic.mic_linear_cross_entropy_backward_kernel_name(mic.handle_for(), code, m, n, k)
    x, w, b = values(1, m, k, dtype=dtype), values(2, n, k, std=2 * k ** -0.5, dtype=dtype), values(3, n, dtype=dtype)
    run(x, w, b, classes(4, m, n, ignored=3 if m > 3 else 0), "sum")


@pytest.mark.parametrize("m,n,k", [(5, 70, 24), (200, 500, 72), (300, 3000, 64), (70, 300, 33)])
@pytest.mark.parametrize("dtype", [F32, BF16])
def test_pitches_and_alignments(m, n, k, dtype):
    def apart(t, pad, start):
        r, c = t.shape
        v = torch.full((start + r * (c + pad) + 3,), float("nan"), dtype=dtype, device=DEV).as_strided((r, c), (c + pad, 1), start)
        return v.copy_(t)

    x, w = values(1, m, k, dtype=dtype), values(2, n, k, std=2 * k ** -0.5, dtype=dtype)
    target = classes(3, m, n)
    for px, sx, pw, sw in ((3, 1, 0, 0), (0, 0, 5, 1), (8, 8, 16, 8), (1, 3, 2, 1)):
        run(apart(x, px, sx), apart(w, pw, sw), None, target, "mean")


def test_leading_dimensions():
    x, w = values(1, 4, 6, 40), values(2, 30, 40)
    target = classes(3, 24, 30)
    one = mic.linear_cross_entropy(x, w, target.reshape(4, 6), reduction="none")
    two = mic.linear_cross_entropy(x.reshape(24, 40), w, target, reduction="none")
    assert one.loss.shape == one.lse.shape == (4, 6) and torch.equal(one.loss.reshape(-1), two.loss)
    dl = values(4, 4, 6)
    g1 = mic.linear_cross_entropy_backward(dl, x, w, target.reshape(4, 6), one.lse)
    g2 = mic.linear_cross_entropy_backward(dl.reshape(-1), x.reshape(24, 40), w, target, two.lse)
    assert g1[0].shape == x.shape and torch.equal(g1[0].reshape(24, 40), g2[0]) and torch.equal(g1[1], g2[1])


# one size each: logits through memory (few rows; split), in their tiles (bf16, fp32)
KINDS = [(5, 60, 32, BF16), (128, 130, 1024, BF16), (260, 140, 256, BF16), (70, 130, 64, F32)]


@pytest.mark.parametrize("m,n,k,dtype", KINDS)
def test_rows_without_a_target(m, n, k, dtype):
    """Their logits, infinite or no numbers, reach neither the loss nor any gradient; without rows both are 0."""
    x, w, b = values(1, m, k, dtype=dtype), values(2, n, k, dtype=dtype), values(3, n, dtype=dtype)
    target = classes(4, m, n, ignored=2)
    got, grads = run(x, w, b, target, "mean")
    assert not grads[0][::2].any()
    x2 = x.clone()
    x2[::2] = 3e38                                           # logits overflow: lse is no number or infinite there
    other = mic.linear_cross_entropy(x2, w, target, bias=b)
    assert torch.equal(other.loss, got.loss) and not other.lse[::2].isfinite().any()
    dx, dw, db = mic.linear_cross_entropy_backward(torch.tensor(1.25, device=DEV), x2, w, target, other.lse, bias=b, count=other.count)
    assert torch.equal(dx, grads[0]) and torch.equal(dw, grads[1]) and torch.equal(db, grads[2])
    none = torch.full_like(target, -100)
    for reduction in ("mean", "sum", "none"):
        r = mic.linear_cross_entropy(x, w, none, bias=b, reduction=reduction)
        assert not r.loss.any()
        dl = torch.ones(m if reduction == "none" else 1, device=DEV)
        for g in mic.linear_cross_entropy_backward(dl, x, w, none, r.lse, bias=b, count=r.count):
            assert not g.any()


@pytest.mark.parametrize("m,n,k,dtype", KINDS)
def test_other_ignore_index(m, n, k, dtype):
    """A class can be the one that marks rows without a target."""
    x, w = values(1, m, k, dtype=dtype), values(2, n, k, dtype=dtype)
    run(x, w, None, classes(4, m, n), "mean", ignore_index=n - 1)
    run(x, w, None, classes(4, m, n), "none", ignore_index=0)


@pytest.mark.parametrize("m,n,k,dtype", KINDS)
def test_masked_classes(m, n, k, dtype):
    """A bias of -infinity, or of the type's lowest value, takes classes out: all others as if those were not there."""
    x, w, b = values(1, m, k, dtype=dtype), values(2, n, k, std=k ** -0.5, dtype=dtype), values(3, n, dtype=dtype)
    keep = torch.arange(n, device=DEV) % 3 != 1
    target = torch.arange(n, device=DEV)[keep][classes(4, m, int(keep.sum()))]
    index = torch.cumsum(keep, 0) - 1
    want = T.cross_entropy(x, w[keep], b[keep], index[target], "none")
    for low in (float("-inf"), torch.finfo(dtype).min):
        masked = torch.where(keep, b, torch.full_like(b, low))
        got = mic.linear_cross_entropy(x, w, target, bias=masked, reduction="none")
        T.check(got.loss, want["loss"], "loss")
        T.check(got.lse, want["lse"], "lse")
        dl = values(5, m)
        dx, dw, db = mic.linear_cross_entropy_backward(dl, x, w, target, got.lse, bias=masked)
        ref = T.cross_entropy_backward(dl, x, w[keep], b[keep], index[target], got.lse, None)
        T.check(dx, ref[0], "dx")
        T.check(dw[keep], ref[1], "dw")
        T.check(db[keep], ref[2], "dbias")
        assert not dw[~keep].any() and not db[~keep].any()
    # a target that is taken out
    out = torch.full_like(target, 1)
    got = mic.linear_cross_entropy(x, w, out, bias=torch.where(keep, b, torch.full_like(b, float("-inf"))), reduction="none")
    assert bool((got.loss == float("inf")).all())


@pytest.mark.parametrize("m,n,k,dtype", KINDS)
def test_no_class_left(m, n, k, dtype):
    x, w = values(1, m, k, dtype=dtype), values(2, n, k, dtype=dtype)
    b = torch.full((n,), float("-inf"), dtype=dtype, device=DEV)
    target = classes(3, m, n)
    got = mic.linear_cross_entropy(x, w, target, bias=b, reduction="none")
    assert bool((got.lse == float("-inf")).all()) and bool((got.loss == float("inf")).all())
    for g in mic.linear_cross_entropy_backward(values(4, m), x, w, target, got.lse, bias=b):
        assert not g.any()


@pytest.mark.parametrize("m,n,k,dtype", KINDS)
def test_targets_that_are_no_class(m, n, k, dtype):
    """Their rows' losses and gradients are no numbers, no other row changes."""
    x, w = values(1, m, k, dtype=dtype), values(2, n, k, dtype=dtype)
    target = classes(3, m, n)
    clean = mic.linear_cross_entropy(x, w, target, reduction="none")
    dl = values(4, m)
    dx0, _, _ = mic.linear_cross_entropy_backward(dl, x, w, target, clean.lse)
    for wrong in (n, -1, -(1 << 40), 1 << 40, (1 << 32) + 1):
        bad = target.clone()
        bad[1] = wrong
        got = mic.linear_cross_entropy(x, w, bad, reduction="none")
        assert bool(got.loss[1].isnan()) and int(got.loss.isnan().sum()) == 1 and torch.equal(got.lse, clean.lse)
        assert bool(mic.linear_cross_entropy(x, w, bad).loss.isnan())
        dx, dw, _ = mic.linear_cross_entropy_backward(dl, x, w, bad, got.lse)
        assert bool(dx[1].isnan().all()) and dw.isnan().all()
        dx[1] = dx0[1]
        assert torch.equal(dx, dx0)


@pytest.mark.parametrize("m,n,k,dtype", KINDS)
def test_far_logits(m, n, k, dtype):
    """Logits of some hundreds, most exponentials nothing; a loss near 0 where the target is far ahead."""
    x, w = values(1, m, k, std=30.0, dtype=dtype), values(2, n, k, std=4 * k ** -0.5, dtype=dtype)
    run(x, w, None, classes(3, m, n), "none")
    best = (x.double() @ w.double().t()).argmax(1)
    run(x, w, None, best, "none")


@pytest.mark.parametrize("m,n,k", [(512, 20011, 64), (40, 5003, 65), (700, 4096, 128)])
@pytest.mark.parametrize("a", [0.0, 0.1])
def test_targets_are_not_rounded_alike(m, n, k, a):
    """Where every class is as likely, a row's gradient is nearly all its target's share, the same number in every row: it
    must not be off the same way in all of them.

    dz = unit (p' - [target]), unit = goal dloss / count, p' = (p - a / classes) / goal, off the target.  Of -1 + p' bf16
    takes 2^-9 at most, and no more than it has (the nearest number to -1 + p' is no further from it than -1 is); of a p'
    half a step, 2^-8 p', and e^x 2^-8 of p more.  Sums are fp32: 2^-24 a term, at most."""
    x, w, t = values(1, m, k, dtype=BF16), values(2, n, k, std=0.01, dtype=BF16), classes(3, m, n)
    got = mic.linear_cross_entropy(x, w, t, label_smoothing=a)
    dloss = torch.tensor(1.2375, device=DEV)                   # 1.2375 and 0.9 times that lie between numbers of bf16
    dx, dw, _ = mic.linear_cross_entropy_backward(dloss, x, w, t, got.lse, count=got.count, label_smoothing=a)
    x, w, t = x.double().cpu(), w.double().cpu(), t.cpu()
    p = torch.softmax(x @ w.T, 1)
    hit = torch.nn.functional.one_hot(t, n).double()
    goal = 1 - a + a / n
    unit = goal * 1.2375 / m
    share = (p - a / n) / goal
    dz = share - hit * ((1 - a) / goal)
    off = torch.where(hit > 0, torch.minimum(p / goal, torch.tensor(2.0 ** -9)), 2.0 ** -8 * share.abs()) + 2.0 ** -8 * p / goal
    for g, want, by in ((dw, dz.T @ x, off.T @ x.abs() + m * 2.0 ** -24 * (dz.abs().T @ x.abs())),
                        (dx, dz @ w, off @ w.abs() + n * 2.0 ** -24 * (dz.abs() @ w.abs()))):
        apart = (g.double().cpu() - unit * want).abs()
        bound = unit * (2.0 ** -8 * want.abs() + (1 + 2.0 ** -8) * by)
        assert bool((apart <= bound).all()), float((apart / bound).max())


@pytest.mark.parametrize("dtype,m,n,k", [(BF16, 256, 1000, 512), (F32, 40, 500, 64), (BF16, 1024, 17003, 128)])
def test_gradients_of_nothing_and_of_no_number(dtype, m, n, k):
    """A dloss of 0 leaves no gradient; one that is infinite or no number leaves rows without a target theirs, 0."""
    x, w, b = values(1, m, k, dtype=dtype), values(2, n, k, std=2 * k ** -0.5, dtype=dtype), values(3, n, dtype=dtype)
    t = classes(4, m, n, ignored=4)
    got = mic.linear_cross_entropy(x, w, t, bias=b)
    for value in (0.0, float("inf"), float("nan")):
        grads = mic.linear_cross_entropy_backward(torch.tensor(value, device=DEV), x, w, t, got.lse, bias=b, count=got.count)
        if value == 0:
            assert not any(bool(g.any()) for g in grads)
        else:
            assert not bool(grads[0][::4].any()) and not bool(grads[0][1].isfinite().any())


@pytest.mark.parametrize("m,n,k,dtype", KINDS)
def test_what_is_not_needed(m, n, k, dtype):
    x, w, b = values(1, m, k, dtype=dtype), values(2, n, k, dtype=dtype), values(3, n, dtype=dtype)
    target = classes(4, m, n)
    r = mic.linear_cross_entropy(x, w, target, bias=b)
    one = torch.ones((), device=DEV)
    full = mic.linear_cross_entropy_backward(one, x, w, target, r.lse, bias=b, count=r.count)
    for need in ((True, False, False), (False, True, False), (False, False, True), (False, False, False), (True, True, False)):
        got = mic.linear_cross_entropy_backward(one, x, w, target, r.lse, bias=b, count=r.count, need_dx=need[0], need_dw=need[1],
                                                need_dbias=need[2])
        for g, f, wanted in zip(got, full, need):
            assert (g is not None) == wanted and (g is None or torch.equal(g, f))


def test_same_target_for_all_rows():
    x, w = values(1, 700, 64, dtype=BF16), values(2, 2000, 64, std=0.2, dtype=BF16)
    run(x, w, None, torch.full((700,), 1234, device=DEV), "mean")


@pytest.mark.parametrize("m,n,k,dtype", KINDS)
def test_captured_and_replayed(m, n, k, dtype):
    x, w, b = values(1, m, k, dtype=dtype), values(2, n, k, dtype=dtype), values(3, n, dtype=dtype)
    target = classes(4, m, n, ignored=3)
    one = torch.ones((), device=DEV)

    def step():
        r = mic.linear_cross_entropy(x, w, target, bias=b, label_smoothing=0.1)
        return (r.loss, r.lse, r.count) + mic.linear_cross_entropy_backward(one, x, w, target, r.lse, bias=b, count=r.count,
                                                                             label_smoothing=0.1)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        first = step()
    side.synchronize()
    for a, e in zip(first, step()):
        assert torch.equal(a, e)                             # the same bits on another stream
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step()
    for i in range(4):
        x.copy_(values(10 + i, m, k, dtype=dtype))
        target.copy_(classes(20 + i, m, n, ignored=2 + i))
        want = step()
        graph.replay()
        torch.cuda.synchronize()
        for a, e in zip(out, want):
            assert torch.equal(a, e)


@pytest.mark.parametrize("k", [4104, 4101])
def test_offsets_past_32_bits(k):
    """x of more than 2^32 elements, of which only the first and last rows have targets."""
    m, n = (1 << 20) + 5, 40
    x = torch.empty(m, k, dtype=BF16, device=DEV).normal_(generator=torch.Generator(DEV).manual_seed(1))
    w, b = values(2, n, k, std=2 * k ** -0.5, dtype=BF16), values(3, n, dtype=BF16)
    ends = torch.cat([torch.arange(50), torch.arange(m - 50, m)]).to(DEV)
    few = classes(4, 100, n)
    target = torch.full((m,), -100, device=DEV)
    target[ends] = few
    got = mic.linear_cross_entropy(x, w, target, bias=b)
    assert float(got.count) == 100
    want = T.cross_entropy(x[ends], w, b, few, "mean")
    T.check(got.loss, want["loss"], "loss")
    T.check(got.lse[ends], want["lse"], "lse")
    dloss = torch.tensor(1.25, device=DEV)
    dx, dw, db = mic.linear_cross_entropy_backward(dloss, x, w, target, got.lse, bias=b, count=got.count)
    ref = T.cross_entropy_backward(dloss, x[ends], w, b, few, got.lse[ends], got.count)
    for g, r, name in ((dx[ends], ref[0], "dx"), (dw, ref[1], "dw"), (db, ref[2], "dbias")):
        T.check(g, r, name)
    assert not any(bool(dx[r:r + (1 << 18)].any()) for r in range(50, m - 50 - (1 << 18), 1 << 18))


def test_nothing():
    x, w, b = values(1, 0, 16), values(2, 10, 16), values(3, 10)
    target = torch.zeros(0, dtype=torch.int64, device=DEV)
    r = mic.linear_cross_entropy(x, w, target, bias=b)
    assert float(r.loss) == 0 and float(r.count) == 0 and r.lse.shape == (0,)
    assert mic.linear_cross_entropy(x, w, target, reduction="none").loss.shape == (0,)
    dx, dw, db = mic.linear_cross_entropy_backward(torch.ones((), device=DEV), x, w, target, r.lse, bias=b, count=r.count)
    assert dx.shape == (0, 16) and dw.shape == (10, 16) and not dw.any() and not db.any()
    # no features: the bias alone
    for m in (3, 70):
        x0, w0, t = torch.zeros(m, 0, device=DEV), torch.zeros(10, 0, device=DEV), classes(4, m, 10)
        got = mic.linear_cross_entropy(x0, w0, t, bias=b, reduction="none")
        T.check(got.loss, T.cross_entropy(x0, w0, b, t, "none")["loss"], "loss")
        dx, dw, db = mic.linear_cross_entropy_backward(torch.ones(m, device=DEV), x0, w0, t, got.lse, bias=b)
        assert dx.shape == (m, 0) and dw.shape == (10, 0)
        T.check(db, T.cross_entropy_backward(torch.ones(m, device=DEV), x0, w0, b, t, got.lse, None)[2], "dbias")
    # a single row without a leading dimension
    x1, w1 = values(5, 16), values(6, 10, 16)
    one = mic.linear_cross_entropy(x1, w1, torch.tensor(7, device=DEV), reduction="none")
    assert one.loss.shape == () and torch.equal(one.loss, mic.linear_cross_entropy(x1[None], w1, torch.tensor([7], device=DEV)).loss)
    g = mic.linear_cross_entropy_backward(torch.ones((), device=DEV), x1, w1, torch.tensor(7, device=DEV), one.lse)
    assert g[0].shape == (16,) and g[1].shape == (10, 16)


def test_two_streams_at_once():
    """Calls in flight on two streams, and from two threads, have workspaces of their own."""
    import threading

    x, w = [values(s, 300, 128, dtype=BF16) for s in (1, 2)], values(3, 3000, 128, std=0.2, dtype=BF16)
    target = classes(4, 300, 3000)
    one = torch.ones((), device=DEV)

    def step(x):
        r = mic.linear_cross_entropy(x, w, target)
        return (r.loss, r.lse) + mic.linear_cross_entropy_backward(one, x, w, target, r.lse, count=r.count)[:2]

    want = [step(v) for v in x]
    torch.cuda.synchronize()
    got = [None, None]

    def work(i):
        s = torch.cuda.Stream()
        with torch.cuda.stream(s):
            for _ in range(20):
                got[i] = step(x[i])
        s.synchronize()

    threads = [threading.Thread(target=work, args=(i,)) for i in range(2)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    for g, e in zip(got, want):
        for a, b in zip(g, e):
            assert torch.equal(a, b)


def test_refusals():
    x, w, b = values(1, 4, 8), values(2, 5, 8), values(3, 5)
    t = torch.tensor([0, 1, 2, 4], device=DEV)
    ok = dict(x=x, w=w, target=t)
    for bad in (dict(w=w[:, :7]), dict(w=w.to(BF16)), dict(w=w[:0]), dict(w=w[0]), dict(target=t[:3]), dict(target=t.int()),
                dict(target=t.cpu()), dict(target=t.reshape(2, 2)), dict(bias=b[:4]), dict(bias=b.to(BF16)), dict(x=x.double()),
                dict(x=x.cpu()), dict(x=x.t()), dict(reduction="max"), dict(reduction=None), dict(label_smoothing=1.0),
                dict(label_smoothing=-0.1), dict(label_smoothing=float("nan")), dict(label_smoothing=b), dict(ignore_index=0.5),
                dict(ignore_index=True), dict(ignore_index=1 << 63)):
        with pytest.raises((ValueError, TypeError)):
            mic.linear_cross_entropy(**dict(ok, **bad))
    r = mic.linear_cross_entropy(x, w, t)
    ok = dict(dloss=torch.ones((), device=DEV), x=x, w=w, target=t, lse=r.lse)
    for bad in (dict(dloss=torch.ones(3, device=DEV)), dict(dloss=torch.ones((), device=DEV, dtype=BF16)), dict(dloss=torch.ones(())),
                dict(lse=r.lse[:3]), dict(lse=r.lse.double()), dict(count=torch.ones(2, device=DEV)), dict(count=torch.ones(())),
                dict(need_dx=x), dict(need_dw=x), dict(need_dbias=x), dict(w=w[:, :7]), dict(target=t[:2]), dict(bias=b[:1]),
                dict(label_smoothing=2)):
        with pytest.raises((ValueError, TypeError)):
            mic.linear_cross_entropy_backward(**dict(ok, **bad))
