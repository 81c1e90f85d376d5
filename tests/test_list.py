"""Gradient lists: global norm, tensor norms and clipping (mpt_list_*),
against a plain binary64 implementation.

Tolerances.  All terms of a sum of squares are non-negative, so a binary64 sum
of n of them is off by at most n * 2^-53 relative whatever its order; the
square root halves that and adds, with the division, two roundings.  The
coefficient is one binary32 rounding of a binary64 quotient.  Given that
coefficient every output is two or three roundings in a fixed order, which
torch's elementwise products on the CPU do alike: outputs are compared bit
for bit.
"""
import ctypes
import math

import pytest

import loss_scaled_fp32_b200 as lsf

F16, BF16, F32 = "float16", "bfloat16", "float32"


def _dtype(name):
    import torch
    return getattr(torch, name)


# ---------------------------------------------------------------------------
# CPU: refusals that need no device
# ---------------------------------------------------------------------------

def _ws(sizes, types, out_types=None):
    n = len(sizes)
    nb = ctypes.c_size_t()
    rc = lsf.lib().mpt_list_workspace_bytes(
        (ctypes.c_int64 * n)(*sizes), (ctypes.c_int32 * n)(*types),
        None if out_types is None else (ctypes.c_int32 * n)(*out_types), n, ctypes.byref(nb))
    return rc, nb.value


def test_workspace_bytes_and_refusals():
    rc, b = _ws([1000, 0, 3], [0, 1, 2])
    assert rc == 0 and b % 256 == 0
    assert _ws([0], [0])[0] == 0                        # an empty list is a list
    assert _ws([355_000_000], [0])[1] < 1 << 20           # tables, no copy of the gradients
    assert _ws([10], [3])[0] == lsf.MPT_ERR_INVALID_ARG
    assert _ws([10], [0], [-1])[0] == lsf.MPT_ERR_INVALID_ARG
    assert _ws([-1], [0])[0] == lsf.MPT_ERR_INVALID_ARG
    assert _ws([1 << 60], [0])[0] == lsf.MPT_ERR_INVALID_ARG
    L = lsf.lib()
    nb = ctypes.c_size_t()
    one = (ctypes.c_int64 * 1)(5)
    t = (ctypes.c_int32 * 1)(0)
    assert L.mpt_list_workspace_bytes(None, t, None, 1, ctypes.byref(nb)) == lsf.MPT_ERR_INVALID_ARG
    assert L.mpt_list_workspace_bytes(one, None, None, 1, ctypes.byref(nb)) == lsf.MPT_ERR_INVALID_ARG
    assert L.mpt_list_workspace_bytes(one, t, None, 0, ctypes.byref(nb)) == lsf.MPT_ERR_INVALID_ARG
    assert L.mpt_list_workspace_bytes(one, t, None, 1, None) == lsf.MPT_ERR_INVALID_ARG


def test_null_lists_and_host_workspaces_are_refused():
    L = lsf.lib()
    assert L.mpt_list_norm(None, None, 1.0, None, 0.0, 0, None) == lsf.MPT_ERR_INVALID_ARG
    assert L.mpt_list_clip(None, None, None, 1.0, None, 0.0, 0, None) == lsf.MPT_ERR_INVALID_ARG
    assert L.mpt_list_wait(None, None, None) == lsf.MPT_ERR_INVALID_ARG
    assert L.mpt_list_views(None, None, None) == lsf.MPT_ERR_INVALID_ARG
    assert L.mpt_list_destroy(None) == 0
    one, t = (ctypes.c_int64 * 1)(5), (ctypes.c_int32 * 1)(0)
    h = ctypes.c_void_p()
    buf = ctypes.create_string_buffer(1 << 16)
    at = (ctypes.addressof(buf) + 255) // 256 * 256
    rc = L.mpt_list_create(one, t, None, 1, ctypes.c_void_p(at), 1 << 15, ctypes.byref(h))
    assert rc in (lsf.MPT_ERR_WORKSPACE, lsf.MPT_ERR_CUDA) and not h.value
    assert L.mpt_list_create(one, t, None, 1, ctypes.c_void_p(at), 16,
                             ctypes.byref(h)) == lsf.MPT_ERR_WORKSPACE
    assert L.mpt_list_create(one, t, None, 1, ctypes.c_void_p(at + 8), 1 << 15,
                             ctypes.byref(h)) == lsf.MPT_ERR_WORKSPACE
    assert L.mpt_list_create(one, t, None, 1, None, 1 << 15, ctypes.byref(h)) == lsf.MPT_ERR_WORKSPACE


def test_a_stream_of_another_device_is_refused():
    """With a stand-in for the stream and a list that has nothing behind it:
    refused before anything is looked at."""
    import torch
    import types
    lst = lsf.GradList.__new__(lsf.GradList)
    lst.device = torch.device("cuda", 0)
    other = types.SimpleNamespace(device=torch.device("cuda", 1))
    for call in (lambda: lst.norm([], stream=other), lambda: lst.clip([], 1.0, stream=other)):
        with pytest.raises(ValueError, match="stream"):
            call()


def test_wait_makes_the_lists_device_current(monkeypatch):
    """Otherwise a list on the default stream of another device than the
    current one would wait for the current one's."""
    import contextlib
    import torch
    import types
    lst = lsf.GradList.__new__(lsf.GradList)
    lst.device, lst._h = torch.device("cuda", 1), ctypes.c_void_p()
    inside = []

    @contextlib.contextmanager
    def on(device, stream):
        inside.append(device)
        yield
        inside.pop()
    seen = []
    fake = types.SimpleNamespace(mpt_list_wait=lambda *a: seen.append(list(inside)) or 0)
    monkeypatch.setattr(lsf, "_on", on)
    monkeypatch.setattr(lsf, "_stream_ptr", lambda stream, device: ctypes.c_void_p())
    monkeypatch.setattr(lsf, "lib", lambda: fake)
    lst.wait()
    assert seen == [[lst.device]]
    lst._h = None


def test_the_allocator_hears_of_every_stream_that_uses_the_workspace(monkeypatch):
    import contextlib
    import torch
    import types
    lst = lsf.GradList.__new__(lsf.GradList)
    lst.device, lst._h, lst.n, lst.sizes = torch.device("cuda", 0), None, 1, [1]
    lst.dtypes = lst.out_dtypes = [torch.float16]
    lst.workspace, lst._result, lst._streams = torch.zeros(8, dtype=torch.uint8), {}, {16}
    told = []
    monkeypatch.setattr(lsf, "_on", lambda device, stream: contextlib.nullcontext())
    monkeypatch.setattr(lsf, "_used_on", lambda stream, *ts: told.append(stream) if any(t is lst.workspace for t in ts) else None)
    monkeypatch.setattr(lsf, "lib", lambda: types.SimpleNamespace(mpt_list_norm=lambda *a: 0, mpt_list_clip=lambda *a: 0))
    home, other, third = (types.SimpleNamespace(device=lst.device, cuda_stream=k) for k in (16, 32, 48))
    ptrs = lsf.grad_pointers([torch.zeros(1)])
    lst.norm(ptrs, stream=home)
    assert told == []
    lst.norm(ptrs, stream=other)
    lst.clip(ptrs, 1.0, stream=other)
    lst.clip(ptrs, 1.0, stream=third)
    assert told == [other, third]


# ---------------------------------------------------------------------------
# GPU
# ---------------------------------------------------------------------------

def _tensors(sizes, dtypes, seed, shift=0, std=3.0, mean=-8.0):
    """Gradients of log-normal magnitude, each `shift` elements past a 64-byte
    boundary of its own buffer."""
    import torch
    g = torch.Generator().manual_seed(seed)
    out = []
    for n, dt in zip(sizes, dtypes):
        x = torch.exp2(torch.randn(n, generator=g) * std + mean)
        x *= torch.randint(0, 2, (n,), generator=g) * 2 - 1
        room = torch.zeros(n + shift + 16, dtype=_dtype(dt), device="cuda")
        room[shift:shift + n] = x.cuda().to(_dtype(dt))
        out.append(room[shift:shift + n])
    return out


def _check(r, tensors, scale, clip):
    """Compare the result views with the definition; returns (coef, inv)."""
    import torch
    clip = ctypes.c_float(clip).value  # the argument is a binary32
    host = [t.cpu().double() for t in tensors]
    bad = sum(int((~torch.isfinite(x)).sum()) for x in host)
    n = sum(x.numel() for x in host)
    sums = [math.fsum((x * x).tolist()) if torch.isfinite(x).all() else math.inf for x in host]
    rel = n * 2.0 ** -54 + 2.0 ** -51
    for got, s in zip(r["tensor_norms"].tolist(), sums):
        want = math.sqrt(s) / scale
        assert got == want or abs(got - want) <= rel * want, (got, want)
    norm, coef = r["norm"].item(), r["coef"].item()
    assert r["n_nonfinite"].item() == bad and r["found_inf"].item() == (1 if bad else 0)
    if bad:
        assert math.isinf(norm) and coef == 1.0
    else:
        want = math.sqrt(math.fsum(sums)) / scale
        assert abs(norm - want) <= rel * want, (norm, want)
        if clip > 0 and norm > clip:
            assert coef == torch.tensor(clip / norm, dtype=torch.float64).float().item()
        else:
            assert coef == 1.0
    return coef


def _expect(t, coef, inv, dtype):
    x = t.float().cpu()
    if inv != 1.0:
        x = x * inv
    return (x * coef).to(dtype)


def _same(a, b):
    import torch
    a, b = a.cpu(), b.cpu()
    nan = torch.isnan(a) & torch.isnan(b)
    ints = {2: torch.int16, 4: torch.int32}[a.element_size()]
    return bool(((a.view(ints) == b.view(ints)) | nan).all())


LISTS = {
    "one": [1],
    "edges": [1, 7, 8, 9, 31, 32, 33, 255, 256, 257, 511, 513, 4095, 4097],
    "empty": [0, 5, 0, 0, 1000, 0],
    "nothing": [0, 0],
    "flat": [1_000_003],
    "mixed": [300_001, 3, 1, 70_000, 2, 2, 2, 65_536, 1_200_007],
    "many": [(i * 37) % 97 for i in range(6000)],
}


@pytest.mark.gpu
@pytest.mark.parametrize("shift", [0, 1, 3])
@pytest.mark.parametrize("kind", [F16, BF16, F32, "all"])
@pytest.mark.parametrize("name", sorted(LISTS))
def test_norm_and_clip_match_the_definition(name, kind, shift):
    import torch
    sizes = LISTS[name]
    types = [[F16, BF16, F32][i % 3] if kind == "all" else kind for i in range(len(sizes))]
    tensors = _tensors(sizes, types, 5, shift)
    same = lsf.GradList(sizes, [_dtype(t) for t in types])
    scale = 1000.0
    r = same.norm(tensors, scale=scale, clip=1e-4, tensor_norms=True)
    coef = _check(r, tensors, scale, 1e-4)
    # out of place into FP32, unscaled, at another alignment
    wide = lsf.GradList(sizes, [_dtype(t) for t in types], torch.float32)
    guard = [torch.full((n + 8,), 7.0, device="cuda") for n in sizes]
    r = wide.clip(tensors, 1e-4, out=[g[1:1 + n] for g, n in zip(guard, sizes)], scale=scale,
                  unscale=True, tensor_norms=True)
    assert _check(r, tensors, scale, 1e-4) == coef
    inv = torch.tensor(1.0) / torch.tensor(scale)
    for t, g, n in zip(tensors, guard, sizes):
        assert _same(g[1:1 + n], _expect(t, coef, inv, torch.float32))
        assert g[0] == 7.0 and bool((g[1 + n:] == 7.0).all())
    # in place
    want = [_expect(t, coef, 1.0, _dtype(k)) for t, k in zip(tensors, types)]
    r = same.clip(tensors, 1e-4, scale=scale)
    for t, w in zip(tensors, want):
        assert _same(t, w)
    d = same.wait()
    assert d["grad_norm"] == r["norm"].item() and d["clip_coef"] == r["coef"].item() == coef
    same.close()
    wide.close()


@pytest.mark.gpu
@pytest.mark.parametrize("kind,out", [(F16, BF16), (BF16, F16), (F32, F16), (F32, BF16), (F16, F16), (BF16, F32)])
def test_every_output_type(kind, out):
    import torch
    sizes = [10_001, 17, 4096]
    tensors = _tensors(sizes, [kind] * 3, 6, shift=2)
    pair = lsf.GradList(sizes, _dtype(kind), _dtype(out))
    outs = [torch.zeros(n, dtype=_dtype(out), device="cuda") for n in sizes]
    r = pair.clip(tensors, 0.01, out=outs, tensor_norms=True)
    coef = _check(r, tensors, 1.0, 0.01)
    assert coef < 1.0
    for t, o in zip(tensors, outs):
        assert _same(o, _expect(t, coef, 1.0, _dtype(out)))


@pytest.mark.gpu
@pytest.mark.parametrize("value", [math.inf, -math.inf, math.nan])
@pytest.mark.parametrize("kind", [F16, BF16, F32])
def test_overflow_leaves_the_gradients(kind, value):
    import torch
    sizes = [5000, 3, 40_000]
    tensors = _tensors(sizes, [kind] * 3, 7, shift=1)
    tensors[2][39_999] = value
    tensors[2][7] = value
    before = [t.clone() for t in tensors]
    lst = lsf.GradList(sizes, _dtype(kind))
    r = lst.clip(tensors, 1e-6, tensor_norms=True)
    assert r["n_nonfinite"].item() == 2
    _check(r, before, 1.0, 1e-6)
    for t, b in zip(tensors, before):
        assert _same(t, b)


@pytest.mark.gpu
def test_extreme_magnitudes_and_repeatability():
    """FP32 squares beyond binary32 at both ends; the same bits each time."""
    import torch
    for mag in (3e38, 1e-40):
        x = torch.full((70_001,), mag, device="cuda")
        lst = lsf.GradList([70_001], torch.float32)
        r = lst.norm([x], tensor_norms=True)
        _check(r, [x], 1.0, 0.0)
    y = _tensors([2_000_001], [F32], 8)
    lst = lsf.GradList([2_000_001], torch.float32)
    first = lst.norm(y)["norm"].item()
    for _ in range(3):
        assert lst.norm(y)["norm"].item() == first


@pytest.mark.gpu
def test_within_the_limit_nothing_is_written_in_place():
    import torch
    sizes = [1000, 33]
    tensors = _tensors(sizes, [F16, F16], 9)
    tensors[0][5] = -0.0
    before = [t.clone() for t in tensors]
    lst = lsf.GradList(sizes, torch.float16)
    assert lst.clip(tensors, 1e9)["coef"].item() == 1.0
    assert lst.clip(tensors, 0.0)["coef"].item() == 1.0      # clip <= 0: off
    for t, b in zip(tensors, before):
        assert _same(t, b)
    out = [torch.ones_like(t) for t in tensors]
    lst.clip(tensors, 1e9, out=out)                          # elsewhere: a copy
    for t, o in zip(tensors, out):
        assert _same(t, o)


@pytest.mark.gpu
def test_device_scale_streams_and_graphs():
    """S read on the device when the work runs; a call on another stream; a
    captured call replayed on new gradients."""
    import torch
    sizes = [30_000, 5, 1024]
    tensors = _tensors(sizes, [F16] * 3, 10)
    outs = [torch.zeros(n, device="cuda") for n in sizes]
    S = torch.full((1,), 256.0, device="cuda")
    lst = lsf.GradList(sizes, torch.float16, torch.float32)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        lst.clip(tensors, 0.001, out=outs, scale=S, unscale=True, tensor_norms=True)
    side.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=side):
        r = lst.clip(tensors, 0.001, out=outs, scale=S, unscale=True, tensor_norms=True)
    for k, s in enumerate((256.0, 64.0)):
        for t, f in zip(tensors, _tensors(sizes, [F16] * 3, 20 + k)):
            t.copy_(f)
        S.fill_(s)
        g.replay()
        torch.cuda.synchronize()
        coef = _check(r, tensors, s, 0.001)
        for t, o in zip(tensors, outs):
            assert _same(o, _expect(t, coef, 1.0 / s, torch.float32))
    # the captured table stays while others come and go
    kept = [_tensors(sizes, [F16] * 3, 30 + k) for k in range(6)]  # six tables: no address comes twice
    for other in kept:
        lst.norm(other)
    torch.cuda.synchronize()
    g.replay()
    torch.cuda.synchronize()
    _check(r, tensors, 64.0, 0.001)
    # a capture with a new table is refused, and records nothing
    fresh = _tensors(sizes, [F16] * 3, 40)
    g2 = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g2, stream=side):
        with pytest.raises(lsf.MptError) as e:
            lst.norm(fresh)
    assert e.value.code == lsf.MPT_ERR_INVALID_ARG


@pytest.mark.gpu
def test_refusals():
    import torch
    lst = lsf.GradList([100, 50], torch.float16)
    room = torch.zeros(400, dtype=torch.float16, device="cuda")
    a, b = room[0:100], room[200:250]

    def code(fn):
        with pytest.raises(lsf.MptError) as e:
            fn()
        return e.value.code

    bad = lsf.MPT_ERR_INVALID_ARG
    assert code(lambda: lst.norm([a, b], scale=0.0)) == bad
    assert code(lambda: lst.norm([a, b], scale=math.nan)) == bad
    assert code(lambda: lst.clip([a, b], math.inf)) == bad
    # outputs on one another, on another gradient, shifted on their own
    assert code(lambda: lst.clip([a, b], 1.0, out=[room[100:200], room[150:200]])) == bad
    assert code(lambda: lst.clip([a, b], 1.0, out=[room[150:250], room[300:350]])) == bad
    assert code(lambda: lst.clip([a, b], 1.0, out=[room[1:101], b])) == bad
    # the same tensor twice is a norm, but no clipping in place
    twin = lsf.GradList([100, 100], torch.float16)
    a.fill_(2.0)
    assert twin.norm([a, a])["norm"].item() == math.sqrt(800.0)
    assert code(lambda: twin.clip([a, a], 1.0)) == bad
    ptrs = lsf.grad_pointers([a, b])
    ptrs[1] = None
    assert code(lambda: lst.norm(ptrs)) == bad
    ptrs[1] = b.data_ptr() + 1
    assert code(lambda: lst.norm(ptrs)) == bad
    for args in (([a],), ([a, b.float()],), ([a, room[200:300:2]],), ([a, b.cpu()],), ([b, a],)):
        with pytest.raises(ValueError):
            lst.norm(*args)
    with pytest.raises(ValueError):
        lst.norm([a, b], scale=torch.ones(1, dtype=torch.float64, device="cuda"))
    with pytest.raises(ValueError):
        lsf.GradList([3], torch.float64)
    with pytest.raises(ValueError):
        lsf.GradList([3], torch.float16, torch.float32).clip([a[:3]], 1.0)
    assert lst.norm([a, b])["found_inf"].item() == 0      # still usable


@pytest.mark.gpu
def test_clip_then_step_is_the_step_that_clips():
    """A list clipped in place and stepped without clipping moves the master
    as one step with clipping does, but for the clipped gradients' FP16
    rounding (half a step of 2^-10 of each, times lr)."""
    import torch
    sizes = [5000, 129]
    S, clip, lr = 2.0 ** 10, 0.001, 0.5  # a norm of about 0.007: clipped
    grads = _tensors(sizes, [F16] * 2, 11, mean=-4.0, std=1.0)
    opts = [lsf.MPT(sizes, lsf.Config()) for _ in range(2)]
    for o in opts:
        o.refresh_half()
    whole = opts[0].step([g.clone() for g in grads], S, lr, 0.0, 0.0, clip)
    exact = [g.double() / S * whole["clip_coef"] for g in grads]
    lst = lsf.GradList(sizes, torch.float16)
    r = lst.clip(grads, clip, scale=S)
    assert whole["clipped"] == 1 and abs(r["norm"].item() - whole["grad_norm"]) <= 1e-12 * whole["grad_norm"]
    assert r["coef"].item() == whole["clip_coef"]
    part = opts[1].step(grads, S, lr, 0.0, 0.0, 0.0)
    assert part["found_inf"] == 0
    for i in range(2):
        step = lr * exact[i].abs()
        # FP16 rounding of the clipped gradient: relative 2^-11, or half the
        # smallest subnormal (2^-25, unscaled by S); then three FP32 roundings
        far = step * (2.0 ** -11 + 2.0 ** -21) + lr * 2.0 ** -25 / S
        assert bool(((opts[0].master(i) - opts[1].master(i)).double().abs() <= far).all())
    for o in opts:
        o.close()


@pytest.mark.gpu
@pytest.mark.parametrize("explicit", [True, False])
def test_a_list_dropped_while_its_call_runs_keeps_its_workspace(explicit):
    """A call on another stream than the list's own, the list dropped at once:
    its workspace is not handed out again before the call is done."""
    import torch
    sizes = [40_000, 7]
    tensors = _tensors(sizes, [F16] * 2, 41)
    want = [t.clone() for t in tensors]
    twin = lsf.GradList(sizes, torch.float16)
    coef = twin.clip(want, 1e-4)["coef"].item()
    assert coef < 1.0
    side = torch.cuda.Stream()
    lst = lsf.GradList(sizes, torch.float16)
    lst.clip(tensors, 1e9)                        # nothing to clip; the pointers are on the device now
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        torch.cuda._sleep(200_000_000)            # some 0.1 s
    kept = lst.workspace.data_ptr()
    if explicit:
        lst.clip(tensors, 1e-4, stream=side)
    else:
        with torch.cuda.stream(side):
            lst.clip(tensors, 1e-4)
    done = side.record_event()
    nbytes = lst.workspace.numel()
    lst = None
    running = not done.query()                    # (unless dropping the list has waited for it)
    again = [torch.full((nbytes,), 255, dtype=torch.uint8, device="cuda") for _ in range(4)]
    assert not running or all(x.data_ptr() != kept for x in again)
    torch.cuda.synchronize()
    for t, w in zip(tensors, want):
        assert _same(t, w)


@pytest.mark.gpu
def test_closing_waits_for_the_copy_of_a_new_table():
    import torch
    tensors = _tensors([1000], [F16], 42)
    lst = lsf.GradList([1000], torch.float16)
    torch.cuda.synchronize()
    torch.cuda._sleep(100_000_000)
    before = torch.cuda.current_stream().record_event()
    r = lst.norm(tensors, tensor_norms=True)
    lst.close()
    assert before.query()
    _check(r, tensors, 1.0, 0.0)


@pytest.mark.gpu
def test_waiting_inside_a_capture_is_refused():
    """The capture goes on, and the list stays usable."""
    import torch
    tensors = _tensors([1000], [F16], 43)
    lst = lsf.GradList([1000], torch.float16)
    lst.norm(tensors)
    x = torch.zeros(4, device="cuda")
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        x.add_(1.0)
        r = lst.norm(tensors, tensor_norms=True)
        with pytest.raises(lsf.MptError) as e:
            lst.wait()
        assert e.value.code == lsf.MPT_ERR_INVALID_ARG
    g.replay()
    torch.cuda.synchronize()
    assert x[0].item() == 1.0
    _check(r, tensors, 1.0, 0.0)
    assert lst.wait()["grad_norm"] == r["norm"].item()


@pytest.mark.gpu
def test_a_list_that_goes_during_a_capture_leaves_it_alone():
    import torch
    tensors = _tensors([1000], [F16], 44)
    lst = lsf.GradList([1000], torch.float16)
    lst.norm(tensors)
    x = torch.zeros(4, device="cuda")
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        x.add_(1.0)
        lst.close()
        x.add_(1.0)
    g.replay()
    torch.cuda.synchronize()
    assert x[0].item() == 2.0


@pytest.mark.gpu
def test_a_workspace_that_is_still_written_by_its_last_owner():
    """The allocator hands out memory in stream order: what the stream's earlier
    work still writes there comes before the list's tables."""
    import torch
    sizes = [40_000, 7]
    tensors = _tensors(sizes, [F16] * 2, 45)
    nbytes = lsf.GradList(sizes, torch.float16).workspace.numel()
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        x = torch.empty(nbytes, dtype=torch.uint8, device="cuda")
        at = x.data_ptr()
        torch.cuda._sleep(200_000_000)            # some 0.1 s
        x.fill_(0)
        x = None
        lst = lsf.GradList(sizes, torch.float16)
        assert lst.workspace.data_ptr() == at
        r = lst.norm(tensors, tensor_norms=True)
    torch.cuda.synchronize()
    _check(r, tensors, 1.0, 0.0)


@pytest.mark.gpu
@pytest.mark.parametrize("kind,bits", [(F16, 0x7C01), (BF16, 0x7F81), (F32, 0x7F800001)])
def test_gradients_that_are_left_are_not_rewritten(kind, bits):
    """Signalling NaN of a payload that widening and rounding change: the bits
    stay where an overflow or the limit leaves the gradients, in place."""
    import torch
    ints = {2: torch.int16, 4: torch.int32}[_dtype(kind).itemsize]
    (x,) = _tensors([70_001], [kind], 46)
    x.view(ints)[69_998] = bits
    x.view(ints)[5] = bits
    before = x.view(ints).clone()
    lst = lsf.GradList([70_001], _dtype(kind))
    assert lst.clip([x], 1e-6)["n_nonfinite"].item() == 2
    assert torch.equal(x.view(ints), before)
