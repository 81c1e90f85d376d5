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
    assert ws(**big, **none) < ws(**big)
    assert ws(n=0) < 4096
    nb = ctypes.c_size_t()
    assert L.mpt_xent_workspace_bytes(None, ctypes.byref(nb)) == lsf.MPT_ERR_INVALID_ARG
    assert L.mpt_xent_workspace_bytes(ctypes.byref(_args(d=9)), ctypes.byref(nb)) == lsf.MPT_ERR_INVALID_ARG


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
    a = (H.abs() @ W.abs().t()).max() if n else torch.tensor(0.0)
    live = t != IGNORE
    at = torch.where(live, t, 0)
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
    e = float(2 * (d / 16 + 16) * acc * a + zmax * 2.0 ** -21 + 2.0 ** -20 + v * 2.0 ** -30)
    small = 2.0 ** -40 * g if kind == torch.float16 else 0.0
    least = 2.0 ** -25 if kind == torch.float16 else 0.0
    dh, dw = dz @ W, dz.t() @ H
    tol_dh = (dz.abs() @ W.abs()) * (u + 2 * e + (v / 16 + 64) * acc) + u * dh.abs() * 1.01 + least + small * W.abs().sum(0)
    tol_dw = (dz.abs().t() @ H.abs()) * (u + 2 * e + (n / 16 + 64) * acc) + u * dw.abs() * 1.01 + least + \
        small * H.abs().sum(0)
    return dict(loss=loss.sum() / by, token_loss=loss, lse=lse, n=k, dh=dh, dw=dw, e=e, tol_dh=tol_dh, tol_dw=tol_dw)


def _close(got, want, tol, what):
    far = (got.double() - want).abs() - tol
    assert bool((far <= 0).all()), (what, float(far.max()), float((got.double() - want).abs().max()))


def _check(r, ref):
    e = ref["e"]
    _close(r.lse, ref["lse"], e + ref["lse"].abs() * 2.0 ** -23, "lse")
    _close(r.token_loss, ref["token_loss"], 2 * e + ref["token_loss"].abs() * 2.0 ** -23, "token_loss")
    _close(r.loss, ref["loss"], (2 * e + ref["loss"].abs() * 2.0 ** -23) * max(1.0, ref["n"] * 1.0
                                                                             if ref["loss"] > 1e6 else 1.0), "loss")
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
