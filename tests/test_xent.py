"""Softmax cross entropy of a head and its loss-scaled gradients (mpt_xent),
against the definition in binary64.

Tolerances, from the arithmetic of the call (u = 2^-11 or 2^-8, half a step
of the 16-bit type):
  z     products of 16-bit values are exact; their binary32 sums, K = 16 at a
        time, are off by at most (d/16 + 16) 2^-23 A, A = max sum |h w|.
  loss  an exponential's argument adds |z| 2^-22 and the exponential 2^-21;
        positive terms keep that relative error through their sum (v / 64
        additions of 2^-24 in a row at most), so with
          e = 2 (d/16 + 16) 2^-23 A + max|z| 2^-21 + 2^-20 + v 2^-30
        lse is off by e, loss by 2e (and by half a binary32 step).
  dz    p is off by e relative, then rounded to 16 bits once (u); below the
        type's normal range (2^-14 / 2^15 in binary16) by 2^-25 / 2^15.
  dH    sum |dz||w| (u + 2e) for that, the sum itself as z's, and its own
        rounding: u |dH| (or half the smallest subnormal); dW likewise.
"""
import ctypes
import math

import pytest

import loss_scaled_fp32_b200 as lsf

IGNORE = -100


# ---------------------------------------------------------------------------
# CPU: refusals that need no device
# ---------------------------------------------------------------------------

def _args(**kw):
    a = lsf.XentArgs()
    assert lsf.lib().mpt_xent_args_init(ctypes.byref(a)) == 0
    good = dict(n=10, v=20, d=16, hidden=1 << 20, ld_hidden=16, weight=2 << 20, ld_weight=16,
                targets=3 << 20, loss=4 << 20, grad_hidden=5 << 20, ld_grad_hidden=16,
                grad_weight=6 << 20, ld_grad_weight=16)
    for k, v in (good | kw).items():
        setattr(a, k, v)
    return a


def test_defaults():
    a = lsf.XentArgs()
    assert lsf.lib().mpt_xent_args_init(ctypes.byref(a)) == 0
    assert (a.type, a.target_bytes, a.ignore_index, a.reduction, a.scale) == (lsf.MPT_F16, 8, -100, 0, 1.0)
    assert lsf.lib().mpt_xent_args_init(None) == lsf.MPT_ERR_INVALID_ARG


def test_refusals_before_any_work():
    """None of these addresses is touched: the call returns before it queues."""
    L = lsf.lib()
    ws = ctypes.c_void_p(256)

    def run(a, size=1 << 40, at=ws):
        return L.mpt_xent(ctypes.byref(a), at, size, None)

    bad = [dict(n=-1), dict(v=0), dict(d=0), dict(d=12), dict(d=4), dict(n=1 << 25), dict(v=1 << 25),
           dict(type=lsf.MPT_F32), dict(type=9), dict(target_bytes=2), dict(reduction=2),
           dict(hidden=None), dict(hidden=(1 << 20) + 8), dict(ld_hidden=8), dict(ld_hidden=17),
           dict(weight=None), dict(weight=(2 << 20) + 2), dict(ld_weight=15), dict(targets=None),
           dict(targets=(3 << 20) + 4), dict(loss=None), dict(loss=(4 << 20) + 2),
           dict(token_loss=(7 << 20) + 1), dict(lse=(7 << 20) + 2), dict(n_valid=(7 << 20) + 4),
           dict(grad_hidden=(5 << 20) + 1), dict(ld_grad_hidden=15), dict(ld_grad_weight=8),
           dict(grad_hidden=1 << 20), dict(grad_weight=2 << 20), dict(grad_weight=(5 << 20) + 64),
           dict(grad_weight=(1 << 20) + 128), dict(scale=0.0), dict(scale=-1.0), dict(scale=math.nan),
           dict(scale=math.inf), dict(d_scale=(7 << 20) + 2)]
    for kw in bad:
        assert run(_args(**kw)) == lsf.MPT_ERR_INVALID_ARG, kw
    assert L.mpt_xent(None, ws, 1 << 40, None) == lsf.MPT_ERR_INVALID_ARG
    assert run(_args(), size=100) == lsf.MPT_ERR_WORKSPACE
    assert run(_args(), at=None) == lsf.MPT_ERR_WORKSPACE
    assert run(_args(), at=ctypes.c_void_p(264)) == lsf.MPT_ERR_WORKSPACE


def test_workspace_bytes():
    L = lsf.lib()

    def ws(**kw):
        nb = ctypes.c_size_t()
        assert L.mpt_xent_workspace_bytes(ctypes.byref(_args(**kw)), ctypes.byref(nb)) == 0
        return nb.value

    none = dict(grad_hidden=None, grad_weight=None)
    big = dict(n=8192, v=50257, d=1024, ld_hidden=1024, ld_weight=1024)
    logits = 8192 * 50257 * 2
    assert ws(**big, **none) < logits // 20                # row statistics
    assert ws(**big) < logits                               # a piece of dz and sums of dH
    # never more than a piece of kept logits (256 MB) and dz (half of it)
    assert ws(n=1300, v=50257, d=1024, ld_hidden=1024, ld_weight=1024, grad_hidden=None) < 420 << 20
    assert ws(**big, **none) < ws(**big)
    assert ws(n=0) < 4096
    nb = ctypes.c_size_t()
    assert L.mpt_xent_workspace_bytes(None, ctypes.byref(nb)) == lsf.MPT_ERR_INVALID_ARG
    assert L.mpt_xent_workspace_bytes(ctypes.byref(_args(d=9)), ctypes.byref(nb)) == lsf.MPT_ERR_INVALID_ARG


def test_workspace_of_many_rows():
    """dz of a piece stays within 256 MB whatever the rows are (and grad_weight's
    sums over the cuts, at most 16384 classes, beside it)."""
    L = lsf.lib()

    def ws(**kw):
        nb = ctypes.c_size_t()
        assert L.mpt_xent_workspace_bytes(ctypes.byref(_args(**kw)), ctypes.byref(nb)) == 0
        return nb.value
    for n in (9000, 20_000, 70_000, 1 << 20, 1 << 24):
        for v in (500, 50257):
            size = dict(n=n, v=v, d=64, ld_hidden=64, ld_weight=64, grad_hidden=None)
            extra = ws(**size) - ws(**size, grad_weight=None)
            assert extra <= (256 << 20) + (16384 * 64 * 4 if n > 16384 else 0) + 4096, (n, v, extra)


# ---------------------------------------------------------------------------
# GPU
# ---------------------------------------------------------------------------

def _inputs(n, v, d, kind, seed, ignored=0.2, sure=20.0, std=0.05):
    import torch
    g = torch.Generator().manual_seed(seed)
    w = torch.randn(v, d, generator=g) * std
    t = torch.randint(0, v, (n,), generator=g)
    h = torch.randn(n, d, generator=g)
    h += torch.rand(n, 1, generator=g) * sure * torch.nn.functional.normalize(w[t], dim=1)
    t[torch.rand(n, generator=g) < ignored] = IGNORE
    dt = getattr(torch, kind)
    return h.to(dt).cuda(), w.to(dt).cuda(), t.cuda()


def _reference(h, w, t, scale, mean=True):
    """Results in binary64 and how far a result may be from them."""
    import torch
    kind = h.dtype
    H, W = h.double(), w.double()
    n, d = H.shape
    v = W.shape[0]
    z = H @ W.t()
    a = float((H.abs() @ W.abs().t()).max()) if n else 0.0
    live = t != IGNORE
    at = torch.where(live, t, 0).long()
    lse = torch.logsumexp(z, 1)
    loss = torch.where(live, lse - z.gather(1, at[:, None])[:, 0], 0.0)
    k = int(live.sum())
    by = max(k, 1) if mean else 1
    g = scale / by
    dz = torch.exp(z - lse[:, None])
    # p_t - 1 = -(sum of the others): a sure row's would cancel even in binary64
    rows = torch.arange(n, device=h.device)
    dz[rows, at] = 0.0
    dz[rows, at] = -dz.sum(1)
    dz *= live[:, None] * g
    u = torch.finfo(kind).eps / 2
    acc = 2.0 ** -23
    zmax = float(z.abs().max()) if n else 0.0
    e = 2 * (d / 16 + 16) * acc * a + zmax * 2.0 ** -21 + 2.0 ** -20 + v * 2.0 ** -30
    small = 2.0 ** -40 * g if kind == torch.float16 else 0.0
    least = 2.0 ** -25 if kind == torch.float16 else 0.0
    dh, dw = dz @ W, dz.t() @ H
    tol_dh = (dz.abs() @ W.abs()) * (u + 2 * e + (v / 16 + 64) * acc) + u * dh.abs() * 1.01 + least + small * W.abs().sum(0)
    tol_dw = (dz.abs().t() @ H.abs()) * (u + 2 * e + (n / 16 + 64) * acc) + u * dw.abs() * 1.01 + least + \
        small * H.abs().sum(0)
    return dict(loss=loss.sum() / by, token_loss=loss, lse=lse, n=k, dh=dh, dw=dw, e=e, tol_dh=tol_dh, tol_dw=tol_dw,
                rows=1 if mean else k)


def _close(got, want, tol, what):
    far = (got.double() - want).abs() - tol
    assert bool((far <= 0).all()), (what, float(far.max()), float((got.double() - want).abs().max()))


def _check(r, ref):
    e = ref["e"]
    _close(r.lse, ref["lse"], e + ref["lse"].abs() * 2.0 ** -23, "lse")
    _close(r.token_loss, ref["token_loss"], 2 * e + ref["token_loss"].abs() * 2.0 ** -23, "token_loss")
    # a mean is off by no more than its rows, a sum by all of them together
    _close(r.loss, ref["loss"], ref["rows"] * 2 * e + ref["loss"].abs() * 2.0 ** -22, "loss")
    assert r.n_valid.item() == ref["n"]
    if isinstance(r, lsf.XentGrad):
        if r.grad_hidden is not None:
            _close(r.grad_hidden, ref["dh"], ref["tol_dh"], "grad_hidden")
        if r.grad_weight is not None:
            _close(r.grad_weight, ref["dw"], ref["tol_dw"], "grad_weight")


SHAPES = [(1, 1, 8), (1, 2, 64), (2, 3, 8), (5, 257, 72), (127, 255, 64), (128, 256, 128), (129, 513, 136),
          (64, 1000, 520), (300, 5003, 264), (1000, 777, 1024), (70, 50257, 96),
          (1, 999, 2056), (2, 50257, 256), (3, 5001, 1000), (4, 33, 504), (4, 300, 12000), (1, 300, 12000)]


@pytest.mark.gpu
@pytest.mark.parametrize("kind", ["float16", "bfloat16"])
@pytest.mark.parametrize("shape", SHAPES, ids=lambda s: "x".join(map(str, s)))
def test_loss_and_gradients_match_the_definition(shape, kind):
    n, v, d = shape
    h, w, t = _inputs(n, v, d, kind, 3)
    scale = 16.0 * n if kind == "float16" else 1.0
    ref = _reference(h, w, t, scale)
    _check(lsf.xent_loss(h, w, t), ref)
    _check(lsf.xent_grad(h, w, t, scale=scale), ref)


@pytest.mark.gpu
@pytest.mark.parametrize("n", [3, 40, 300])
def test_sum_int32_targets_and_one_gradient_at_a_time(n):
    import torch
    h, w, t = _inputs(n, 500, 128, "float16", 5)
    ref = _reference(h, w, t, 4.0, mean=False)
    t32 = t.to(torch.int32)
    _check(lsf.xent_loss(h, w, t32, reduction="sum"), ref)
    r = lsf.xent_grad(h, w, t32, scale=4.0, reduction="sum", grad_weight=None)
    assert r.grad_weight is None
    _check(r, ref)
    r = lsf.xent_grad(h, w, t32, scale=4.0, reduction="sum", grad_hidden=False)
    assert r.grad_hidden is None
    _check(r, ref)
    r = lsf.xent_grad(h, w, t32, scale=4.0, reduction="sum", grad_hidden=None, grad_weight=None)
    assert r.grad_hidden is None and r.grad_weight is None
    _check(r, ref)


@pytest.mark.gpu
@pytest.mark.parametrize("kind", ["float16", "bfloat16"])
def test_several_pieces_and_cut_sums(kind):
    """dz of 4000 x 40000 takes two pieces of the vocabulary, the second one
    short; 200 x 40000 one piece with dH's sum cut in parts."""
    for n, v, d in ((4000, 40000, 64), (200, 40001, 136)):
        h, w, t = _inputs(n, v, d, kind, 6)
        scale = 16.0 * n if kind == "float16" else 1.0
        _check(lsf.xent_grad(h, w, t, scale=scale), _reference(h, w, t, scale))


@pytest.mark.gpu
@pytest.mark.parametrize("n", [2, 50, 200])
def test_rows_with_gaps_and_unaligned_gradients(n):
    import torch
    v, d = 700, 200
    h0, w0, t = _inputs(n, v, d, "float16", 7)
    scale = 16.0 * n
    ref = _reference(h0, w0, t, scale)

    def gap(x, ld, shift=0):
        room = torch.full((x.shape[0] * ld + 64,), 3.0, dtype=x.dtype, device="cuda")
        out = room[shift:shift + x.shape[0] * ld].view(x.shape[0], ld)[:, :d]
        out.copy_(x)
        return out, room
    h, _ = gap(h0, 264)
    w, _ = gap(w0, 208)
    for ld, shift in ((d, 0), (d + 8, 8), (d + 1, 0), (d + 8, 1), (d + 3, 5)):
        gh, room_h = gap(h0, ld, shift)
        gw, room_w = gap(w0, ld, shift)
        r = lsf.xent_grad(h, w, t, scale=scale, grad_hidden=gh, grad_weight=gw)
        assert r.grad_hidden is gh and r.grad_weight is gw
        _check(r, ref)
        for room, rows in ((room_h, n), (room_w, v)):      # nothing beside the rows is written
            keep = torch.ones_like(room, dtype=torch.bool)
            keep[shift:shift + rows * ld].view(rows, ld)[:, :d] = False
            assert bool((room[keep] == 3.0).all())


def test_the_row_distance_of_one_row_is_not_looked_at():
    """A row cut out of a matrix of any width is a matrix like any other."""
    import torch
    cpu = torch.device("cpu")
    x = torch.zeros(3, 1001, dtype=torch.float16)
    assert lsf._rows(x[1:2, :64], "hidden", torch.float16, cpu) == 64
    assert lsf._rows(x[:, :64], "hidden", torch.float16, cpu) == 1001
    assert lsf._rows(torch.zeros(1, 64, dtype=torch.float16).expand(1, 64), "hidden", torch.float16, cpu) == 64


@pytest.mark.gpu
def test_one_row_of_a_matrix_of_any_width():
    import torch
    h, w, t = _inputs(1, 300, 64, "float16", 32, ignored=0.0)
    ref = _reference(h, w, t, 16.0)
    room = [torch.full((2, 1001), 3.0, dtype=torch.float16, device="cuda") for _ in range(2)]
    room[0][:1, :64] = h
    gh = room[1][:1, :64]
    r = lsf.xent_grad(room[0][:1, :64], w, t, scale=16.0, grad_hidden=gh)
    _check(r, ref)
    assert r.grad_hidden is gh and bool((room[1][:, 64:] == 3.0).all()) and bool((room[1][1:] == 3.0).all())
    one = torch.full((2, 1001), 3.0, dtype=torch.float16, device="cuda")[:1, :64]   # a head of one class
    one.copy_(w[:1])
    r = lsf.xent_grad(h, one, torch.zeros_like(t))
    assert r.loss.item() == 0.0 and not r.grad_weight.any()


@pytest.mark.gpu
@pytest.mark.parametrize("shape", [(3, 5003, 200), (50, 5003, 200), (200, 5003, 200), (4000, 33536 + 70, 72)],
                         ids=lambda s: "x".join(map(str, s)))
def test_unaligned_gradients_of_cut_sums_and_pieces(shape):
    """dH in five parts, written row by row at odd distances; the last shape has
    a second piece of two blocks, fewer than the parts, whose dW starts in the
    middle of an unaligned matrix."""
    import torch
    n, v, d = shape
    h, w, t = _inputs(n, v, d, "float16", 33)
    ref = _reference(h, w, t, 16.0 * n)
    for extra, shift in ((1, 0), (3, 5), (8, 8), (8, 1)):
        ld = d + extra
        rooms = [torch.full((rows * ld + 16,), 3.0, dtype=torch.float16, device="cuda") for rows in (n, v)]
        gh, gw = (room[shift:shift + rows * ld].view(rows, ld)[:, :d] for room, rows in zip(rooms, (n, v)))
        _check(lsf.xent_grad(h, w, t, scale=16.0 * n, grad_hidden=gh, grad_weight=gw), ref)
        for room, rows in zip(rooms, (n, v)):
            keep = torch.ones_like(room, dtype=torch.bool)
            keep[shift:shift + rows * ld].view(rows, ld)[:, :d] = False
            assert bool((room[keep] == 3.0).all())


@pytest.mark.gpu
@pytest.mark.parametrize("kind", ["float16", "bfloat16"])
def test_a_last_piece_of_fewer_blocks_than_parts(kind):
    n, v, d = 4000, 33536 + 70, 64
    h, w, t = _inputs(n, v, d, kind, 34)
    scale = 16.0 * n if kind == "float16" else 1.0
    ref = _reference(h, w, t, scale)
    _check(lsf.xent_grad(h, w, t, scale=scale), ref)
    _check(lsf.xent_grad(h, w, t, scale=scale, grad_weight=None), ref)


@pytest.mark.gpu
@pytest.mark.parametrize("n", [1, 4, 60, 300])
def test_nothing_left_to_learn(n):
    """Every row ignored; no row at all."""
    import torch
    h, w, t = _inputs(n, 333, 72, "float16", 8)
    t.fill_(IGNORE)
    r = lsf.xent_grad(h, w, t, scale=1024.0)
    assert r.loss.item() == 0.0 and r.n_valid.item() == 0
    assert not r.token_loss.any() and not r.grad_hidden.any() and not r.grad_weight.any()
    ref = _reference(h, w, t, 1.0)
    _close(r.lse, ref["lse"], ref["e"] + ref["lse"].abs() * 2.0 ** -23, "lse")
    r = lsf.xent_grad(h[:0], w, t[:0], scale=2.0, grad_weight=torch.ones_like(w))
    assert r.loss.item() == 0.0 and r.n_valid.item() == 0 and r.grad_hidden.shape == (0, 72)
    assert not r.grad_weight.any()
    r = lsf.xent_loss(h[:0], w, t[:0])
    assert r.loss.item() == 0.0 and r.token_loss.numel() == 0


@pytest.mark.gpu
@pytest.mark.parametrize("n", [2, 50, 300])
@pytest.mark.parametrize("bad", [-1, 1000, 1 << 40, -(1 << 62)])
def test_a_target_that_is_no_class_poisons_the_result(n, bad):
    import torch
    h, w, t = _inputs(n, 1000, 64, "float16", 9, ignored=0.0)
    t[n // 2] = bad
    r = lsf.xent_grad(h, w, t)
    assert math.isnan(r.loss.item()) and r.n_valid.item() == n
    nan = torch.isnan(r.token_loss)
    assert nan[n // 2] and int(nan.sum()) == 1
    assert bool(torch.isnan(r.grad_hidden[n // 2]).all()) and bool(torch.isnan(r.grad_weight).all())
    assert not bool(torch.isnan(r.grad_hidden[:n // 2]).any())


@pytest.mark.gpu
@pytest.mark.parametrize("n", [1, 4, 100, 260])
def test_an_ignored_index_that_is_a_class(n):
    import torch
    h, w, t = _inputs(n, 64, 64, "bfloat16", 10, ignored=0.0)
    t[:] = torch.arange(n, device="cuda") % 3
    ref = _reference(h, w, torch.where(t == 1, IGNORE, t), 1.0)
    _check(lsf.xent_grad(h, w, t, ignore_index=1), ref)


@pytest.mark.gpu
@pytest.mark.parametrize("n", [2, 90, 300])
def test_extreme_logits(n):
    """Logits of some thousands (nothing overflows), and a class that every row
    excludes: a weight row that makes its logit -inf."""
    import torch
    h, w, t = _inputs(n, 600, 64, "bfloat16", 11, ignored=0.0, sure=0.0, std=100.0)
    r = lsf.xent_loss(h, w, t)
    _check(r, _reference(h, w, t, 1.0))
    assert float(r.token_loss.max()) > 1000.0
    h, w, t = _inputs(n, 600, 64, "float16", 12, ignored=0.0)
    h[:, 0] = 1.0
    w[7] = 0.0
    w[7, 0] = -math.inf
    t[t == 7] = 8
    keep = torch.arange(600, device="cuda") != 7
    ref = _reference(h, w[keep], t - (t > 7).long(), 1.0)
    _check(lsf.xent_loss(h, w, t), ref)
    t[0] = 7                                      # and one row whose target it is
    assert lsf.xent_loss(h, w, t).token_loss[0].item() == math.inf
    # rows that are nothing but -inf, and NaN in a row: NaN, there alone
    w[:] = 0.0
    w[:, 0] = -math.inf
    assert math.isnan(lsf.xent_loss(h, w, t).token_loss[0].item())
    h, w, t = _inputs(n, 600, 64, "float16", 13, ignored=0.0)
    h[1, 5] = math.nan
    r = lsf.xent_loss(h, w, t)
    assert math.isnan(r.token_loss[1].item()) and int(torch.isnan(r.token_loss).sum()) == 1


@pytest.mark.gpu
@pytest.mark.parametrize("shape", [(2, 600, 64), (90, 600, 64), (300, 600, 64), (6000, 1000, 136)],
                         ids=lambda s: "x".join(map(str, s)))
@pytest.mark.parametrize("low", [-math.inf, -3e4])
def test_a_target_far_below_the_others(low, shape):
    """lse keeps its places, and a target's logit of -inf leaves the row an
    infinite loss and finite probabilities.  (Logits kept and multiplied again;
    the column of the low logit is left out of A and of the largest |z|: its
    products are 0 but for one, which is exact.)"""
    import torch
    n, v, d = shape
    h, w, t = _inputs(n, v, d, "float16", 23, ignored=0.0, std=0.3)
    h[:, 0] = 1.0
    w[:, 0] = 0.0
    w[7] = 0.0
    w[7, 0] = low
    t[t == 7] = 8
    t[n // 2] = 7
    keep = torch.arange(v, device="cuda") != 7
    # without class 7, whose probability is 0 (the row's target: any other)
    t0 = torch.where(t == 7, 0, t - (t > 7).long())
    ref = _reference(h, w[keep], t0, 16.0 * n)
    e = ref["e"]
    r = lsf.xent_grad(h, w, t, scale=16.0 * n, grad_hidden=True)
    _close(r.lse, ref["lse"], e + ref["lse"].abs() * 2.0 ** -23, "lse")
    row = n // 2
    if low == -math.inf:
        assert r.token_loss[row].item() == math.inf and r.loss.item() == math.inf
    else:
        want = ref["lse"][row] - low
        _close(r.token_loss[row], want, 2 * e + want * 2.0 ** -23, "token_loss")
    # dW: the row adds p h to the others (its stand-in class 0 took h away) and
    # -h to class 7
    H = h.double()
    dw = torch.zeros(v, d, dtype=torch.float64, device="cuda")
    dw[keep] = ref["dw"]
    dw[0] += 16.0 * H[row]
    dw[7] = -16.0 * H[row]
    tol = torch.zeros_like(dw)
    tol[keep] = ref["tol_dw"]
    tol[7] = 16.0 * H[row].abs() * 2.0 ** -9
    tol[0] += 16.0 * H[row].abs() * 2.0 ** -9
    _close(r.grad_weight, dw, tol, "grad_weight")
    # dH of the other rows; of this one beside the column of the low weight,
    # where the other classes' sum is 0 and this class adds -(low)
    others = torch.arange(n, device="cuda") != row
    _close(r.grad_hidden[others][:, 1:], ref["dh"][others][:, 1:], ref["tol_dh"][others][:, 1:], "grad_hidden")
    if low != -math.inf:
        W = w.double()
        dh = ref["dh"][row] + 16.0 * W[0]
        assert bool(((r.grad_hidden[row].double() - dh)[1:].abs() <=
                     (ref["tol_dh"][row] + 16.0 * W[0].abs() * 2.0 ** -9)[1:]).all())


@pytest.mark.gpu
@pytest.mark.parametrize("n", [2, 90, 300])
def test_a_logit_of_plus_infinity_is_never_sure(n):
    """log(sum exp z) - z_t is inf - inf where the target's logit is +inf: NaN,
    not a loss of 0 that would hide the overflow."""
    import torch
    h, w, t = _inputs(n, 600, 64, "float16", 24, ignored=0.0)
    w[:, 0] = 0.0
    w[7] = 0.0
    w[7, 0] = math.inf
    h[:, 0] = -1.0                                # -inf for the other rows
    h[n // 2, 0] = 1.0
    t[t == 7] = 8
    for target in (7, 8):
        t[n // 2] = target
        r = lsf.xent_grad(h, w, t)
        for each in (r.token_loss, r.lse):
            nan = torch.isnan(each)
            assert nan[n // 2] and int(nan.sum()) == 1
        assert math.isnan(r.loss.item())
        assert bool(torch.isnan(r.grad_hidden[n // 2]).all()) and bool(torch.isnan(r.grad_weight).all())


@pytest.mark.gpu
@pytest.mark.parametrize("n,kind", [(400_003, "float16"), (3_000_001, "bfloat16")])
def test_long_sums_over_the_rows(n, kind):
    """dW of rows that all pull one way.  Eight classes of equal logits: dz is
    1/8 or -7/8, exact in 16 bits, so what is left is the sum: in parts of at
    most 16384 rows, where 16 of K lose at most two of the sum's last places
    (2 * 2^-23), the parts added to nearest, and one rounding of the result."""
    import torch
    dt = getattr(torch, kind)
    g = torch.Generator(device="cuda").manual_seed(25)
    h = (1 + torch.rand(n, 8, generator=g, device="cuda")).to(dt)
    w = torch.zeros(8, 8, dtype=dt, device="cuda")
    t = torch.zeros(n, dtype=torch.int64, device="cuda")
    r = lsf.xent_grad(h, w, t, scale=64.0)
    want = h.double().sum(0) * (8.0 / n) * torch.tensor([-7.0] + [1.0] * 7, dtype=torch.float64, device="cuda")[:, None]
    rel = torch.finfo(dt).eps / 2 * 1.01 + 1024 * 2 * 2.0 ** -23 + (n / 8192) * 2.0 ** -24 + 2.0 ** -20
    _close(r.grad_weight, want, want.abs() * rel, "grad_weight")
    assert not r.grad_hidden.any()


@pytest.mark.gpu
@pytest.mark.parametrize("kind", ["float16", "bfloat16"])
@pytest.mark.parametrize("shape", [(20_000, 700, 72), (20_000, 700, 1024), (33_000, 14_000, 64), (16_641, 300, 136)],
                         ids=lambda s: "x".join(map(str, s)))
def test_more_rows_than_one_cut(shape, kind):
    """Two and three cuts of the rows: logits multiplied again, logits kept,
    and two pieces of the vocabulary; a last cut of other length."""
    n, v, d = shape
    h, w, t = _inputs(n, v, d, kind, 26)
    scale = 16.0 * n if kind == "float16" else 1.0
    ref = _reference(h, w, t, scale)
    _check(lsf.xent_grad(h, w, t, scale=scale), ref)
    _check(lsf.xent_grad(h, w, t, scale=scale, grad_weight=None), ref)
    _check(lsf.xent_grad(h, w, t.int(), scale=scale, grad_hidden=None), ref)


@pytest.mark.gpu
def test_cuts_write_rows_with_gaps():
    import torch
    n, v, d = 16_400, 300, 72
    h, w, t = _inputs(n, v, d, "float16", 27)
    ref = _reference(h, w, t, 16.0 * n)
    room_h = torch.full((n * 75 + 8,), 3.0, dtype=torch.float16, device="cuda")
    room_w = torch.full((v * 73 + 8,), 3.0, dtype=torch.float16, device="cuda")
    gh, gw = room_h[1:1 + n * 75].view(n, 75)[:, :d], room_w[3:3 + v * 73].view(v, 73)[:, :d]
    _check(lsf.xent_grad(h, w, t, scale=16.0 * n, grad_hidden=gh, grad_weight=gw), ref)
    for room, shift, rows, ld in ((room_h, 1, n, 75), (room_w, 3, v, 73)):
        keep = torch.ones_like(room, dtype=torch.bool)
        keep[shift:shift + rows * ld].view(rows, ld)[:, :d] = False
        assert bool((room[keep] == 3.0).all())


@pytest.mark.gpu
@pytest.mark.parametrize("kind", ["float16", "bfloat16"])
@pytest.mark.parametrize("shape", [(128, 50257, 64), (100, 60001, 72), (2500, 3001, 72), (6000, 1000, 136),
                                   (1100, 8111, 264), (700, 20000, 512)], ids=lambda s: "x".join(map(str, s)))
def test_logits_multiplied_again_in_one_piece(shape, kind):
    """Many logits of narrow rows: quicker to multiply again than to keep."""
    n, v, d = shape
    h, w, t = _inputs(n, v, d, kind, 20)
    scale = 16.0 * n if kind == "float16" else 1.0
    _check(lsf.xent_grad(h, w, t, scale=scale), _reference(h, w, t, scale))


@pytest.mark.gpu
@pytest.mark.parametrize("kind", ["float16", "bfloat16"])
def test_logits_multiplied_again_are_those_of_the_loss(kind):
    """Logits of about 2000, all of one sign: what the tensor cores drop adds up
    in each, and only cancels against the row's lse where the backward pass
    makes the same logits again.  Rows of a large call (multiplied again)
    against the same rows of a small one (logits kept).  Both round the same
    dz but for the places of lse (2 steps of 2^-23) and for what that moves
    across a rounding to 16 bits (2 u); their sums over v differ in order, and
    each result is rounded once."""
    import torch
    n, v, d, few = 4200, 16400, 8192, 200
    g = torch.Generator(device="cuda").manual_seed(22)
    dt = getattr(torch, kind)
    h = (1 + 0.01 * torch.randn(n, d, generator=g, device="cuda")).to(dt)
    w = (0.25 + 0.01 * torch.randn(v, d, generator=g, device="cuda")).to(dt)
    t = torch.randint(0, v, (n,), generator=g, device="cuda")
    again = lsf.xent_grad(h, w, t, scale=64.0, reduction="sum", grad_weight=None)
    kept = lsf.xent_grad(h[:few], w, t[:few], scale=64.0, reduction="sum")
    W = w.double()
    z = h[:few].double() @ W.t()
    p = 64.0 * torch.softmax(z, 1)
    size = p @ W.abs() + 64.0 * W[t[:few]].abs()
    assert float(z.min()) > 1900.0
    u = torch.finfo(dt).eps / 2
    tol = size * (2 * u + float(kept.lse.max()) * 2.0 ** -22 + 2 * (v / 16 + 64) * 2.0 ** -23) + \
        2 * u * kept.grad_hidden.double().abs() + 2.0 ** -24
    _close(again.grad_hidden[:few], kept.grad_hidden.double(), tol, "grad_hidden")


@pytest.mark.gpu
def test_few_rows_of_the_largest_vocabulary():
    """2^24 classes: too many logits to keep, even of four rows."""
    h, w, t = _inputs(4, 1 << 24, 8, "bfloat16", 21, ignored=0.0)
    _check(lsf.xent_grad(h, w, t), _reference(h, w, t, 1.0))


@pytest.mark.gpu
def test_small_probabilities_survive_binary16():
    """dz below binary16's range times S / n: rows with 2^-24-sized
    probabilities still pull their weight."""
    import torch
    n, v, d = 256, 300, 64
    h, w, t = _inputs(n, v, d, "float16", 14, ignored=0.0, sure=0.0, std=0.01)
    h[:, 0] = 4.0
    w[:, 0] = -1.0
    w[:5, 0] = 3.0                                # the other 295 classes: exp(-16) = 1e-7 each
    t[:] = torch.arange(n, device="cuda") % 5
    ref = _reference(h, w, t, 2.0 ** 14)
    r = lsf.xent_grad(h, w, t, scale=2.0 ** 14)
    _check(r, ref)
    tail = ref["dw"][5:, 0]
    assert float(tail.abs().min()) > 0 and bool((r.grad_weight[5:, 0] != 0).all())
    assert bool(((r.grad_weight[5:, 0].double() - tail).abs() <= 0.01 * tail.abs() + 2.0 ** -24).all())


@pytest.mark.gpu
def test_gradients_against_differences():
    """Directional differences of the binary64 loss: exact to about
    eps^2 |third derivative| (1e-8 here); the gradients' own tolerance is
    what a direction can gather."""
    import torch
    h, w, t = _inputs(40, 200, 64, "bfloat16", 15)
    ref = _reference(h, w, t, 1.0)
    r = lsf.xent_grad(h, w, t)
    g = torch.Generator(device="cuda").manual_seed(0)

    def loss(H, W):
        live = t != IGNORE
        z = H @ W.t()
        return (torch.logsumexp(z, 1) - z.gather(1, torch.where(live, t, 0)[:, None])[:, 0])[live].mean()
    H, W, eps = h.double(), w.double(), 1e-4
    for x, grad, tol in ((H, r.grad_hidden, ref["tol_dh"]), (W, r.grad_weight, ref["tol_dw"])):
        for _ in range(5):
            d = torch.randn(x.shape, generator=g, device="cuda", dtype=torch.float64)
            diff = (loss(H + eps * d, W) - loss(H - eps * d, W)) if x is H else (loss(H, W + eps * d) - loss(H, W - eps * d))
            assert abs(float(diff / (2 * eps) - (grad.double() * d).sum())) <= float((tol * d.abs()).sum()) + 1e-6


@pytest.mark.gpu
@pytest.mark.parametrize("n", [4, 100, 700])
def test_same_bits_each_time_on_streams_and_in_graphs(n):
    import torch
    v, d = 9000, 192
    h, w, t = _inputs(n, v, d, "float16", 16)
    S = torch.full((1,), 64.0, device="cuda")
    first = lsf.xent_grad(h, w, t, scale=S)

    def same(a, b):
        return all(torch.equal(x, y) for x, y in zip(a, b))
    # two calls at once, on streams of their own
    streams = [torch.cuda.Stream() for _ in range(2)]
    for s in streams:
        s.wait_stream(torch.cuda.current_stream())
    rs = []
    for k in range(6):
        with torch.cuda.stream(streams[k % 2]):
            rs.append(lsf.xent_grad(h, w, t, scale=S))
    rs.append(lsf.xent_grad(h, w, t, scale=S, stream=streams[0]))
    torch.cuda.synchronize()
    assert all(same(first, r) for r in rs)
    # captured, replayed on other inputs and another S
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=streams[0]):
        r = lsf.xent_grad(h, w, t, scale=S)
    h2, w2, t2 = _inputs(n, v, d, "float16", 17)
    h.copy_(h2)
    w.copy_(w2)
    t.copy_(t2)
    S.fill_(256.0)
    g.replay()
    torch.cuda.synchronize()
    assert same(r, lsf.xent_grad(h2, w2, t2, scale=256.0))
    _check(r, _reference(h2, w2, t2, 256.0))


@pytest.mark.gpu
@pytest.mark.parametrize("n", [2, 40])
def test_offsets_beyond_31_bits(n):
    """A head of 2.2e9 values: its last rows are read and written."""
    import torch
    v, d = 270_000, 8192
    w = torch.zeros(v, d, dtype=torch.bfloat16, device="cuda")
    g = torch.Generator(device="cuda").manual_seed(1)
    w[-2000:] = torch.randn(2000, d, generator=g, device="cuda").mul_(0.02).bfloat16()
    h = torch.randn(n, d, generator=g, device="cuda").bfloat16()
    t = torch.arange(v - n, v, device="cuda")
    r = lsf.xent_grad(h, w, t)
    H, W = h.double(), w[-2000:].double()
    z = H @ W.t()                                   # the other 268000 logits are 0
    lse = torch.logaddexp(torch.logsumexp(z, 1), torch.tensor(math.log(v - 2000.0), device="cuda"))
    loss = lse - z[:, -n:].diagonal()
    # e as above with A <= |h| |w| (Cauchy-Schwarz), max|z| <= 12
    e = 2 * (d / 16 + 16) * 2.0 ** -23 * float(H.norm(dim=1).max() * W.norm(dim=1).max()) + 12 * 2.0 ** -21 + \
        2.0 ** -20 + v * 2.0 ** -30
    _close(r.token_loss, loss, 2 * e + loss * 2.0 ** -23, "token_loss")
    dz = torch.exp(z - lse[:, None])
    dz[torch.arange(n, device="cuda"), torch.arange(2000 - n, 2000, device="cuda")] -= 1.0
    dz /= n
    u = 2.0 ** -8
    tol = (dz.abs().t() @ H.abs()) * (u + 2 * e + 66 * 2.0 ** -23) + u * 1.01 * (dz.t() @ H).abs()
    _close(r.grad_weight[-2000:], dz.t() @ H, tol, "grad_weight")
    want = dz @ W
    _close(r.grad_hidden, want, (dz.abs() @ W.abs()) * (u + 2 * e + (v / 16 + 64) * 2.0 ** -23) + u * 1.01 * want.abs(),
           "grad_hidden")


def test_the_hook_that_lets_waits_run_out():
    L = lsf.lib()
    assert L.mpt_debug_xent_give_up(8) == lsf.MPT_ERR_INVALID_ARG
    assert L.mpt_debug_xent_give_up(7) == 0 and L.mpt_debug_xent_give_up(0) == 0


@pytest.mark.gpu
@pytest.mark.parametrize("passes", [1, 2, 4, 7])
@pytest.mark.parametrize("shape", [(100, 60001, 72), (700, 9000, 192), (300, 900, 1024)], ids=lambda s: "x".join(map(str, s)))
def test_waits_that_run_out_end_the_call(shape, passes):
    """One CTA to a tile, two, and logits kept: every block gives up where it
    would wait, ends what it has in flight and leaves; the loss is NaN, and the
    next call is whole."""
    import torch
    n, v, d = shape
    h, w, t = _inputs(n, v, d, "float16", 28)
    good = lsf.xent_grad(h, w, t, scale=16.0 * n)
    for _ in range(4):
        assert lsf.lib().mpt_debug_xent_give_up(passes) == 0
        r = lsf.xent_grad(h, w, t, scale=16.0 * n)
        torch.cuda.synchronize()
        if passes != 2 or d < 1000:                # (2: kept logits are not multiplied again)
            assert math.isnan(r.loss.item())
    r = lsf.xent_grad(h, w, t, scale=16.0 * n)
    assert all(torch.equal(a, b) for a, b in zip(r, good))


@pytest.mark.gpu
@pytest.mark.parametrize("passes", [1, 2, 4])
@pytest.mark.parametrize("shape", [(100, 60001, 72), (700, 9000, 192), (300, 900, 1024), (17_000, 700, 72),
                                   (4000, 40_000, 64)], ids=lambda s: "x".join(map(str, s)))
def test_no_gradient_looks_whole_after_a_wait_that_ran_out(shape, passes):
    """Sums cut, results final, logits kept, cuts of the rows, two pieces."""
    import torch
    n, v, d = shape
    if passes == 2 and shape == (300, 900, 1024):
        return                                     # kept logits are not multiplied again
    h, w, t = _inputs(n, v, d, "float16", 29)
    for kw in (dict(), dict(grad_hidden=None), dict(grad_weight=None)):
        good = lsf.xent_grad(h, w, t, scale=16.0 * n, **kw)
        grads = {k: torch.full_like(x, 3.0) for k, x in good._asdict().items() if k.startswith("grad") and x is not None}
        assert lsf.lib().mpt_debug_xent_give_up(passes) == 0
        r = lsf.xent_grad(h, w, t, scale=16.0 * n, **(kw | grads))
        assert math.isnan(r.loss.item())
        if passes == 1:
            assert bool(torch.isnan(r.token_loss[t != IGNORE]).all()) and bool(torch.isnan(r.lse).all())
        for name, x in grads.items():
            nan = torch.isnan(x)
            assert bool(nan.any()) if passes == 4 else bool(nan.all()), name


@pytest.mark.gpu
def test_a_step_skips_after_a_wait_that_ran_out():
    import torch
    v, d, n = 1000, 128, 200
    h, w0, t = _inputs(n, v, d, "float16", 30)
    opt = lsf.MPT([v * d], lsf.Config())
    opt.master(0).copy_(w0.float().flatten())
    opt.refresh_half()
    opt.set_scaler_state(64.0)
    grad = torch.zeros(v * d, dtype=torch.float16, device="cuda")
    before = opt.master(0).clone()
    for passes in (1, 4):
        assert lsf.lib().mpt_debug_xent_give_up(passes) == 0
        opt.head_grad(0, h, t, grad_weight=grad.view(v, d))
        opt.step_async([grad], 0.5, 0.0, 0.0)
        assert opt.wait()["found_inf"] == 1
        assert torch.equal(opt.master(0), before)
    opt.head_grad(0, h, t, grad_weight=grad.view(v, d))
    opt.step_async([grad], 0.5, 0.0, 0.0)
    assert opt.wait()["found_inf"] == 0 and not torch.equal(opt.master(0), before)
    opt.close()


def test_refusals_of_the_binding_on_the_cpu():
    import torch
    h, w, t = torch.zeros(4, 16).half(), torch.zeros(8, 16).half(), torch.zeros(4, dtype=torch.int64)
    for fn in (lsf.xent_loss, lsf.xent_grad):
        with pytest.raises(ValueError):
            fn(h, w, t)


@pytest.mark.gpu
def test_a_stream_of_another_device_is_refused():
    """With a stand-in for the stream: refused before it is used at all."""
    import torch
    import types
    h, w, t = _inputs(10, 50, 64, "float16", 31)
    other = types.SimpleNamespace(device=torch.device("cuda", h.device.index + 1))
    with pytest.raises(ValueError, match="stream"):
        lsf.xent_loss(h, w, t, stream=other)
    with pytest.raises(ValueError, match="stream"):
        lsf.xent_grad(h, w, t, stream=other)


@pytest.mark.gpu
def test_refusals_of_the_binding():
    import torch
    h, w, t = _inputs(10, 50, 64, "float16", 18)
    good = dict(hidden=h, weight=w, targets=t)
    for kw in (dict(hidden=h.float()), dict(weight=w.bfloat16()), dict(hidden=h[None]), dict(weight=w[:, :32]),
               dict(hidden=h.t()), dict(targets=t[:9]), dict(targets=t.float()), dict(targets=t.cpu()),
               dict(targets=torch.stack([t, t], 1)[:, 0]), dict(weight=w.cpu()), dict(hidden=h.float(), weight=w.float()),
               dict(reduction="none")):
        with pytest.raises(ValueError):
            lsf.xent_loss(**(good | kw))
    for kw in (dict(grad_hidden=torch.zeros_like(h)[:5]), dict(grad_weight=torch.zeros(50, 64, device="cuda")),
               dict(grad_weight=torch.zeros_like(w).cpu()), dict(scale=torch.ones(2, device="cuda")),
               dict(scale=torch.ones(1))):
        with pytest.raises(ValueError):
            lsf.xent_grad(**(good | kw))
    for kw in (dict(hidden=torch.zeros(10, 60, device="cuda").half(), weight=torch.zeros(50, 60, device="cuda").half()),
               dict(hidden=torch.zeros(10, 65, device="cuda").half()[:, 1:]), dict(scale=0.0), dict(scale=math.inf),
               dict(grad_hidden=h), dict(grad_weight=w)):
        with pytest.raises(lsf.MptError) as e:
            lsf.xent_grad(**(good | kw))
        assert e.value.code == lsf.MPT_ERR_INVALID_ARG, kw
    _check(lsf.xent_grad(**good), _reference(h, w, t, 1.0))     # and the good call still works


# ---------------------------------------------------------------------------
# the operators together, as a training step uses them
# ---------------------------------------------------------------------------

@pytest.mark.gpu
def test_head_loss_norm_and_step_together():
    """Loss and gradients from the handle's FP16 copy and device scale, the
    norm of the gradients, the step; then an S that overflows FP16 makes the
    gradients inf, the list finds it, and the step skips and halves S."""
    import torch
    v, d, n = 1000, 128, 200
    h, w0, t = _inputs(n, v, d, "float16", 19)
    opt = lsf.MPT([v * d, d], lsf.Config())
    opt.master(0).copy_(w0.float().flatten())
    opt.refresh_half()
    opt.set_scaler_state(2.0 ** 12)
    grads = [torch.zeros(v * d, dtype=torch.float16, device="cuda"),
             torch.full((d,), 0.25, dtype=torch.float16, device="cuda")]
    lst = lsf.GradList([v * d, d], torch.float16)
    assert torch.equal(opt.w16(0), w0.flatten())
    r = opt.head_grad(0, h, t, grad_weight=grads[0].view(v, d))
    norms = lst.norm(grads, scale=opt.device_scale(), tensor_norms=True)
    opt.step_async(grads, 0.5, 0.0, 0.0)
    res = opt.wait()
    ref = _reference(h, w0, t, 2.0 ** 12)
    _check(r, ref)
    assert res["found_inf"] == 0
    got = norms["norm"].item()
    assert abs(got - res["grad_norm"]) <= 1e-12 * got
    assert abs(norms["tensor_norms"][0].item() - float(ref["dw"].norm()) / 2 ** 12) <= float(ref["tol_dw"].norm()) / 2 ** 12
    # the step took this gradient: w - lr g, one rounding each
    want = w0.double().flatten() - 0.5 * grads[0].double() / 2 ** 12
    assert bool(((opt.master(0).double() - want).abs() <= want.abs() * 2.0 ** -23 + 1e-12).all())
    # the loss at the new weights is that of the new FP16 copy
    r2 = opt.head_grad(0, h, t, grad_weight=grads[0].view(v, d))
    _check(r2, _reference(h, opt.w16(0).view(v, d), t, 2.0 ** 12))
    # overflow: dW of some class is about S / n * sum of its rows' hidden
    opt.set_scaler_state(2.0 ** 23)
    before = opt.master(0).clone()
    r = opt.head_grad(0, h, t, grad_weight=grads[0].view(v, d))
    assert math.isfinite(r.loss.item())
    found = lst.norm(grads, scale=opt.device_scale())
    opt.step_async(grads, 0.5, 0.0, 0.0)
    res = opt.wait()
    assert res["found_inf"] == 1 and res["new_scale"] == 2.0 ** 22 and found["found_inf"].item() == 1
    assert found["n_nonfinite"].item() == res["n_nonfinite"] > 0
    assert torch.equal(opt.master(0), before)
    with pytest.raises(ValueError):
        opt.head_grad(0, h[:, :120], t)
    opt.close()
