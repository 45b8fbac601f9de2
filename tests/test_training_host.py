"""Layer norm, dropout and cross entropy without a GPU: refusals, workspaces, and the tests' own formulas against differences."""
import pytest
import torch

import convolution_forward_conv2d_amd as mic
import training_ref as T
from test_feed_forward_host import BAD, BF16, BIG, E4M3, F32, F64, UNSUPPORTED, P, call, handle, status

NORM = "h dtype out rows cols eps x ldx res ldr weight bias y ldy sum lds mean rstd scale".split()
NORM_OK = dict(h=None, dtype=BF16, out=BF16, rows=4, cols=8, eps=1e-5, x=P, ldx=8, res=0, ldr=0, weight=P, bias=0, y=P, ldy=8,
               sum=0, lds=0, mean=0, rstd=0, scale=0)


@pytest.mark.parametrize("change,want", [
    (dict(h=0), BAD), (dict(rows=-1), BAD), (dict(cols=0), BAD), (dict(cols=-1), BAD), (dict(eps=-1.0), BAD),
    (dict(eps=float("nan")), BAD), (dict(x=0), BAD), (dict(weight=0), BAD), (dict(y=0), BAD), (dict(ldx=7), BAD),
    (dict(res=P, ldr=7), BAD), (dict(sum=P, lds=7), BAD), (dict(out=E4M3), BAD), (dict(rstd=P + 2), BAD), (dict(mean=P + 2), BAD),
    (dict(bias=P + 1), BAD), (dict(out=F32), UNSUPPORTED), (dict(dtype=F64, out=F64), UNSUPPORTED),
    (dict(dtype=E4M3, out=E4M3), UNSUPPORTED), (dict(cols=1 << 22, ldx=1 << 22, ldy=1 << 22), UNSUPPORTED)])
def test_norm_refusals(change, want):
    assert call("mic_layer_norm", NORM, dict(NORM_OK, h=handle()), **change) == want


NGRAD = "h dtype rows cols dy lddy sum lds weight mean rstd dsum ldd dx lddx dweight dbias work bytes".split()
NGRAD_OK = dict(h=None, dtype=F32, rows=2000, cols=8, dy=P, lddy=8, sum=P, lds=8, weight=P, mean=P, rstd=P, dsum=0, ldd=0, dx=P,
                lddx=8, dweight=P, dbias=P, work=P, bytes=BIG)


@pytest.mark.parametrize("change,want", [
    (dict(h=0), BAD), (dict(cols=0), BAD), (dict(dy=0), BAD), (dict(sum=0), BAD), (dict(weight=0), BAD), (dict(mean=0), BAD),
    (dict(rstd=0), BAD), (dict(dx=0), BAD), (dict(dsum=P, ldd=7), BAD), (dict(work=0), BAD), (dict(bytes=4), BAD),
    (dict(dweight=P + 2), BAD), (dict(dbias=P + 2), BAD), (dict(dweight=0, work=0), BAD), (dict(dtype=E4M3), UNSUPPORTED),
    (dict(rows=0, cols=1 << 21), UNSUPPORTED)])
def test_norm_backward_refusals(change, want):
    assert call("mic_layer_norm_backward", NGRAD, dict(NGRAD_OK, h=handle()), **change) == want


DROP = "h dtype rows cols p seed offset state x ldx res ldr y ldy".split()
DROP_OK = dict(h=None, dtype=BF16, rows=4, cols=8, p=0.5, seed=1, offset=0, state=0, x=P, ldx=8, res=0, ldr=0, y=P, ldy=8)


@pytest.mark.parametrize("change,want", [
    (dict(h=0), BAD), (dict(rows=-1), BAD), (dict(cols=-1), BAD), (dict(p=-0.1), BAD), (dict(p=1.1), BAD),
    (dict(p=float("nan")), BAD), (dict(x=0), BAD), (dict(y=0), BAD), (dict(x=P + 1), BAD), (dict(ldx=7), BAD), (dict(ldy=7), BAD),
    (dict(res=P, ldr=7), BAD), (dict(state=P + 4), BAD), (dict(dtype=E4M3), UNSUPPORTED), (dict(dtype=F64), UNSUPPORTED),
    (dict(rows=1 << 40), UNSUPPORTED), (dict(rows=1 << 20, cols=1 << 21, ldx=1 << 21, ldy=1 << 21), UNSUPPORTED),
    (dict(ldx=1 << 39), UNSUPPORTED)])
def test_dropout_refusals(change, want):
    assert call("mic_dropout", DROP, dict(DROP_OK, h=handle()), **change) == want


def test_nothing_to_do_is_done():
    assert call("mic_layer_norm", NORM, dict(NORM_OK, h=handle()), rows=0, x=0, y=0, weight=0) == 0
    assert call("mic_layer_norm_backward", NGRAD, dict(NGRAD_OK, h=handle()), rows=0, dweight=0, dbias=0, work=0) == 0
    for n in (dict(rows=0), dict(cols=0)):
        assert call("mic_dropout", DROP, dict(DROP_OK, h=handle()), x=0, y=0, **n) == 0


def test_workspaces():
    # few rows have no partial sums; 1000 rows of 9 columns four side by side, at least three of those to a group
    assert mic.mic_layer_norm_backward_workspace(None, 1, 9) == 0
    assert mic.mic_layer_norm_backward_workspace(None, 1000, 9) == 84 * 9 * 8
    assert status("mic_layer_norm_backward_workspace", None, 4, 4, None) == BAD
    # without a handle the answer serves any number of compute units
    sizes = [(1, 1), (100, 512), (5000, 4096), (5000, 9000), (5000, 20000)]
    assert all(mic.mic_layer_norm_backward_workspace(None, *s) >= mic.mic_layer_norm_backward_workspace(handle(), *s) for s in sizes)


def test_tensor_functions_refuse_before_the_gpu():
    x, w = torch.zeros(4, 8), torch.zeros(8)
    for f, args in ((mic.layer_norm, (x, w)), (mic.layer_norm_backward, (x, x, w, x[:, 0], x[:, 0])), (mic.dropout, (x, 0.5, 1)),
                    (mic.dropout_backward, (x, 0.5, 1)), (mic.linear_cross_entropy, (x, x, x[:, 0].long())),
                    (mic.linear_cross_entropy_backward, (x[0, 0], x, x, x[:, 0].long(), x[:, 0]))):
        with pytest.raises(ValueError, match="GPU"):
            f(*args)
        with pytest.raises(TypeError):
            f(*(a.double() if torch.is_tensor(a) and a.is_floating_point() else a for a in args))


def test_generator():
    """The published known answers of Philox4x32 with ten rounds."""
    def words(lots):
        return [int(lots[2 * i]) | int(lots[2 * i + 1]) << 16 for i in range(4)]

    assert words(T.lots(8, 0, 0)) == [0x6627e8d5, 0xe169c58d, 0xbc57ac4c, 0x9b00dbd8]
    # counter (i / 8, offset) and key seed
    assert words(T.lots(8, 0x299f31d0a4093822, 0x0370734413198a2e, first=8 * 0x85a308d3243f6a88)) == [
        0xd16cfe09, 0x94fdcceb, 0x5001e420, 0x24126ea1]


def differences(f, at, along, h=1e-5):
    """Directional derivative of f by central differences, in float64."""
    return (f(at + h * along) - f(at - h * along)) / (2 * h)


def test_norm_formula_against_differences():
    g = torch.Generator().manual_seed(5)
    s, dy, dsum, v = (torch.randn(3, 17, generator=g, dtype=torch.float64) for _ in range(4))
    w, b, vw = (torch.randn(17, generator=g, dtype=torch.float64) for _ in range(3))

    def value(s, w, b):
        mean = s.mean(1, keepdim=True)
        y = (s - mean) / torch.sqrt((s - mean).square().mean(1, keepdim=True) + 1e-5) * w + b
        return (y * dy).sum() + (s * dsum).sum()

    mean = s.mean(1)
    rstd = 1 / torch.sqrt((s - mean[:, None]).square().mean(1) + 1e-5)
    T.HALF[torch.float64] = 0.0
    try:
        (dx, _), (dw, _), (db, _) = T.layer_norm_backward(dy, s, w, mean, rstd, dsum)
    finally:
        del T.HALF[torch.float64]
    # central differences are off by h^2 f''' / 6 and by 2^-52 |f| / h: below 1e-8 of values of order 10
    assert abs(float((dx * v).sum() - differences(lambda t: value(t, w, b), s, v))) < 1e-6
    assert abs(float((dw * vw).sum() - differences(lambda t: value(s, t, b), w, vw))) < 1e-6
    assert abs(float((db * vw).sum() - differences(lambda t: value(s, w, t), b, vw))) < 1e-6


LOSS = "h dtype red m n k x ldx w ldw bias target ignore smooth loss lse count work bytes".split()
LOSS_OK = dict(h=None, dtype=BF16, red=2, m=4, n=8, k=16, x=P, ldx=16, w=P, ldw=16, bias=0, target=P, ignore=-100, smooth=0.0,
               loss=P, lse=P, count=P, work=P, bytes=BIG)


@pytest.mark.parametrize("change,want", [
    (dict(h=0), BAD), (dict(m=-1), BAD), (dict(n=-1), BAD), (dict(n=0), BAD), (dict(k=-1), BAD), (dict(x=0), BAD), (dict(w=0), BAD),
    (dict(ldx=15), BAD), (dict(ldw=15), BAD), (dict(x=P + 1), BAD), (dict(bias=P + 1), BAD), (dict(target=0), BAD),
    (dict(target=P + 4), BAD), (dict(loss=0), BAD), (dict(loss=P + 2), BAD), (dict(lse=0), BAD), (dict(lse=P + 2), BAD),
    (dict(count=0), BAD), (dict(count=P + 2), BAD), (dict(smooth=1.0), BAD), (dict(smooth=-0.5), BAD),
    (dict(smooth=float("nan")), BAD), (dict(work=0), BAD), (dict(work=P + 8), BAD), (dict(bytes=16), BAD),
    (dict(red=3), UNSUPPORTED), (dict(red=-1), UNSUPPORTED), (dict(dtype=E4M3), UNSUPPORTED), (dict(dtype=F64), UNSUPPORTED),
    (dict(m=1 << 30), UNSUPPORTED), (dict(n=1 << 30), UNSUPPORTED), (dict(ldx=1 << 22), UNSUPPORTED)])
def test_loss_refusals(change, want):
    assert call("mic_linear_cross_entropy", LOSS, dict(LOSS_OK, h=handle()), **change) == want


LGRAD = "h dtype m n k dloss rows x ldx w ldw bias target ignore smooth lse count dx lddx dw lddw db work bytes".split()
LGRAD_OK = dict(h=None, dtype=F32, m=4, n=8, k=16, dloss=P, rows=0, x=P, ldx=16, w=P, ldw=16, bias=0, target=P, ignore=-100,
                smooth=0.0, lse=P, count=0, dx=P, lddx=16, dw=P, lddw=16, db=P, work=P, bytes=BIG)


@pytest.mark.parametrize("change,want", [
    (dict(h=0), BAD), (dict(m=-1), BAD), (dict(n=0), BAD), (dict(dloss=0), BAD), (dict(dloss=P + 2), BAD), (dict(x=0), BAD),
    (dict(w=0), BAD), (dict(ldx=15), BAD), (dict(ldw=15), BAD), (dict(lddx=15), BAD), (dict(lddw=15), BAD), (dict(dx=P + 2), BAD),
    (dict(dw=P + 2), BAD), (dict(db=P + 2), BAD), (dict(bias=P + 2), BAD), (dict(target=0), BAD), (dict(target=P + 4), BAD),
    (dict(lse=0), BAD), (dict(count=P + 2), BAD), (dict(smooth=1.5), BAD), (dict(work=0), BAD), (dict(bytes=16), BAD),
    (dict(dtype=E4M3), UNSUPPORTED), (dict(k=1 << 30), UNSUPPORTED), (dict(lddw=1 << 21), UNSUPPORTED)])
def test_loss_backward_refusals(change, want):
    assert call("mic_linear_cross_entropy_backward", LGRAD, dict(LGRAD_OK, h=handle()), **change) == want


def test_loss_with_nothing_to_do():
    assert call("mic_linear_cross_entropy", LOSS, dict(LOSS_OK, h=handle()), red=0, m=0, x=0, w=0, loss=0) == 0
    assert call("mic_linear_cross_entropy_backward", LGRAD, dict(LGRAD_OK, h=handle()), dx=0, dw=0, db=0, work=0) == 0
    assert call("mic_linear_cross_entropy_backward", LGRAD, dict(LGRAD_OK, h=handle()), m=0, n=0, work=0) == 0


def test_loss_workspaces():
    """The logits of 8192 x 131072 would be 4 GB in fp32; no call holds that much."""
    sizes = [(1, 1, 1), (7, 33, 65), (128, 1000, 4096), (4096, 50021, 4096), (8192, 131072, 4096), (0, 5, 5), (5, 5, 0)]
    fs = ((mic.mic_linear_cross_entropy_workspace, mic.mic_linear_cross_entropy_workspace_aligned),
          (mic.mic_linear_cross_entropy_backward_workspace, mic.mic_linear_cross_entropy_backward_workspace_aligned))
    for any_rows, aligned in fs:
        for dtype in (F32, BF16):
            for m, n, k in sizes:
                size = 4 if dtype == F32 else 2
                most = (1 << 30) + size * (m + min(n, 1 << 19)) * (k + 16) + 4 * m * (k + 8)
                assert 0 <= aligned(None, dtype, m, n, k) <= any_rows(None, dtype, m, n, k) <= 2 * most
                assert aligned(handle(), dtype, m, n, k) <= aligned(None, dtype, m, n, k)
    assert mic.mic_linear_cross_entropy_workspace_aligned(None, BF16, 8192, 131072, 4096) < 8192 * 131072
    for f in fs[0] + fs[1]:
        with pytest.raises(mic.MicError) as e:
            f(None, E4M3, 4, 4, 4)
        assert e.value.status == UNSUPPORTED


def test_loss_formula_against_differences():
    g = torch.Generator().manual_seed(6)
    m, n, k, a = 5, 11, 7, 0.2
    x, w, b = torch.randn(m, k, generator=g).double(), torch.randn(n, k, generator=g).double(), torch.randn(n, generator=g).double()
    vx, vw, vb = (torch.randn(t.shape, generator=g).double() for t in (x, w, b))
    target = torch.tensor([0, 10, -100, 3, 3])
    T.HALF[torch.float64] = 0.0
    try:
        for reduction in ("mean", "sum", "none"):
            weight = torch.randn(m, generator=g) if reduction == "none" else torch.ones(())

            def value(x, w, b):
                return (T.cross_entropy(x, w, b, target, reduction, a=a)["loss"][0] * weight.double()).sum()

            lse = torch.logsumexp(x @ w.t() + b, 1)
            count = torch.tensor(4.0) if reduction == "mean" else None
            (dx, _), (dw, _), (db, _) = T.cross_entropy_backward(weight, x, w, b, target, lse, count, a=a)
            assert abs(float((dx * vx).sum() - differences(lambda t: value(t, w, b), x, vx))) < 1e-6
            assert abs(float((dw * vw).sum() - differences(lambda t: value(x, t, b), w, vw))) < 1e-6
            assert abs(float((db * vb).sum() - differences(lambda t: value(x, w, t), b, vb))) < 1e-6
    finally:
        del T.HALF[torch.float64]
