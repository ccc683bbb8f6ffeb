"""Router, order by expert, dispatch and combine, and their gradients, against
plain implementations in 64 bits; refusals on the CPU, values on a GPU.

Tolerances. Rounding to a type is off by at most eps / 2 of the value (U
below). Weights and p: the argument l - max is exact to 2^-24 of itself, exp
is good to 2 ulp and one division or product follows, so a weight is within
(|l - max| + 8) 2^-23 of itself, below 2^-18 for |l - max| < 24; smaller p
count only absolutely. Gradients of the logits are sums of a few products of
such numbers: 2^-17 of the sum of the terms' absolute values. Rows: dispatch
copies; a combine of k terms is within (k + 1) 2^-24 of the sum of absolute
values before its one rounding; a dot of K terms in fp32 within K 2^-24 of the
sum of absolute values (the true error is far smaller, 32 lanes share it).
"""
import math

import pytest
import torch

from mxfp8_quantization_moe_device_b200 import autograd, binding as mxq

U = {torch.bfloat16: 2.0 ** -8, torch.float32: 2.0 ** -24}
DEV = "cuda"


# ------------------------------------------------------------ plain forms
def ref_route(logits, k, valid=None, renorm=False, gw=None, gl=None):
    """64-bit router: weights, ids, counts, loss and, with gw and gl, the
    gradient and the sum of its terms' absolute values. Rows one by one."""
    T, E = logits.shape
    l = logits.double().cpu()
    ok = torch.ones(T, dtype=torch.bool) if valid is None else valid.cpu().bool()
    w, ids = torch.zeros(T, k, dtype=torch.float64), torch.full((T, k), -1, dtype=torch.int32)
    p, S = torch.zeros(T, E, dtype=torch.float64), torch.zeros(T, dtype=torch.float64)
    bad = torch.zeros(T, dtype=torch.bool)
    for t in range(T):
        if not ok[t]:
            continue
        row = l[t].tolist()
        if any(math.isnan(v) or v == math.inf for v in row):
            bad[t] = True
            p[t], w[t] = math.nan, math.nan
            continue
        live = [e for e in range(E) if row[e] > -math.inf]
        if not live:
            continue
        m = max(row)
        p[t] = torch.tensor([math.exp(v - m) for v in row], dtype=torch.float64)
        p[t] /= p[t].sum()
        best = sorted(live, key=lambda e: (-row[e], e))[:k]
        ids[t, :len(best)] = torch.tensor(best, dtype=torch.int32)
        w[t, :len(best)] = p[t, best]
        S[t] = w[t].sum()
        if renorm:
            w[t] /= S[t]
    counts = torch.tensor([int((ids == e).sum()) for e in range(E)], dtype=torch.int32)
    n = int(ok.sum())
    hb = counts.double() * E / (k * n * n) if n else torch.zeros(E, dtype=torch.float64)
    loss = (hb * p.sum(0)).sum()
    if gw is None and gl is None:
        return w, ids, counts, loss
    gw = torch.zeros(T, k, dtype=torch.float64) if gw is None else gw.double().cpu()
    hb = hb * (0.0 if gl is None else float(gl))
    d, mag = torch.zeros(T, E, dtype=torch.float64), torch.zeros(T, E, dtype=torch.float64)
    for t in range(T):
        if bad[t]:
            d[t] = math.nan
            continue
        h, ha = hb.clone(), hb.abs()
        u = gw[t] * (ids[t] >= 0)
        if renorm and S[t] > 0:
            um = (u.abs() + (u * w[t]).abs().sum()) / S[t]
            u = (u - (u * w[t]).sum()) / S[t]
        else:
            um = u.abs()
        for j in range(k):
            if ids[t, j] >= 0:
                h[ids[t, j]] += u[j]
                ha[ids[t, j]] += um[j]
        d[t] = p[t] * (h - (h * p[t]).sum())
        mag[t] = p[t] * (ha + (ha * p[t]).sum())
    return w, ids, counts, loss, d, mag


def ref_plan(ids, E):
    flat = ids.reshape(-1).tolist()
    order = sorted((e, i) for i, e in enumerate(flat) if 0 <= e < E)
    pos = torch.full((len(flat),), -1, dtype=torch.int32)
    for r, (_, i) in enumerate(order):
        pos[i] = r
    ends, c = [], 0
    for e in range(E):
        c += sum(1 for x in flat if x == e)
        ends.append(c)
    return pos.reshape(ids.shape), torch.tensor(ends, dtype=torch.int32)


def logits_of(T, E, dtype, seed, closed=0, ties=False):
    g = torch.Generator().manual_seed(seed)
    l = torch.randn(T, E, generator=g) * 2.0
    if ties:
        l = (l * 2).round() / 2
        l[l == 0] *= -1.0  # both zeros, equal to each other
    if closed:
        l[:, torch.randperm(E, generator=g)[:closed]] = -math.inf
    return l.to(dtype)


def ids_of(T, E, k, seed, dropped=0.0):
    g = torch.Generator().manual_seed(seed)
    ids = torch.stack([torch.randperm(max(E, k), generator=g)[:k] % E for _ in range(T)]).to(torch.int32) \
        if T else torch.zeros(0, k, dtype=torch.int32)
    ids[torch.rand(T, k, generator=g) < dropped] = -1
    return ids


def near(got, want, tol, what):
    got, want, tol = got.detach().double().cpu(), want.double(), torch.as_tensor(tol, dtype=torch.float64)
    assert got.shape == want.shape, what
    nan = want.isnan()
    assert torch.equal(got.isnan(), nan), f"{what}: NaN in other places"
    over = ((got - want).abs() > tol)[~nan] if tol.dim() else ((got - want).abs()[~nan] > tol)
    assert not bool(over.any()), f"{what}: off by {float((got - want).abs()[~nan].max())}"


# ------------------------------------------------------------ refusals (CPU)
def test_host_checks():
    L = mxq.lib()
    p = 256  # a non-null pointer that is never followed: the checks come first
    assert L.moe_route(p, 0, 4, 0, 0, None, 1, 0, p, p, p, p, None, p, 1 << 20, None) == mxq.ERR_SHAPE
    assert L.moe_route(p, 0, 4, 8, 7, None, 1, 0, p, p, p, p, None, p, 1 << 20, None) == mxq.ERR_SHAPE
    assert L.moe_route(p, 0, 4, 8, 8, None, 9, 0, p, p, p, p, None, p, 1 << 20, None) == mxq.ERR_SHAPE
    assert L.moe_route(p, 0, 4, 8, 8, None, 0, 0, p, p, p, p, None, p, 1 << 20, None) == mxq.ERR_SHAPE
    assert L.moe_route(p, 2, 4, 8, 8, None, 2, 0, p, p, p, p, None, p, 1 << 20, None) == mxq.ERR_UNSUPPORTED
    assert L.moe_route(p, 0, 4, 1025, 1025, None, 2, 0, p, p, p, p, None, p, 1 << 20, None) == mxq.ERR_UNSUPPORTED
    assert L.moe_route(p, 0, 4, 64, 64, None, 33, 0, p, p, p, p, None, p, 1 << 20, None) == mxq.ERR_UNSUPPORTED
    assert L.moe_route(None, 0, 4, 8, 8, None, 2, 0, p, p, p, p, None, p, 1 << 20, None) == mxq.ERR_NULL
    assert L.moe_route(p, 0, 4, 8, 8, None, 2, 0, p, None, p, p, None, p, 1 << 20, None) == mxq.ERR_NULL
    assert L.moe_route(p + 1, 0, 4, 8, 8, None, 2, 0, p, p, p, p, None, p, 1 << 20, None) == mxq.ERR_ALIGN
    assert L.moe_route_backward(p, 0, 4, 8, 8, None, 2, 0, p, p, None, p, p, p, None) == mxq.ERR_NULL
    assert L.moe_route_backward(p, 1, 4, 8, 8, None, 2, 0, p, p, p, p, p, None, None) == mxq.ERR_NULL
    assert L.moe_route_backward(p + 2, 1, 4, 8, 8, None, 2, 0, p, p, p, p, p, p, None) == mxq.ERR_ALIGN
    assert L.moe_route_backward(None, 0, 0, 8, 8, None, 2, 0, None, None, None, None, None, None, None) == mxq.OK
    assert L.moe_dispatch_plan(p, -1, 8, p, p, None, 0, None) == mxq.ERR_SHAPE
    assert L.moe_dispatch_plan(p, 8, 1025, p, p, None, 0, None) == mxq.ERR_UNSUPPORTED
    assert L.moe_dispatch_plan(p, 1 << 31, 8, p, p, None, 0, None) == mxq.ERR_UNSUPPORTED
    assert L.moe_dispatch_plan(p, 8, 8, None, p, None, 0, None) == mxq.ERR_NULL
    assert L.moe_dispatch_plan(p, 100000, 8, p, p, None, 0, None) == mxq.ERR_WORKSPACE
    assert L.moe_dispatch(p, 0, 4, 64, 63, p, 2, p, 4, p, 16, None) == mxq.ERR_SHAPE
    assert L.moe_dispatch(p, 0, 4, 64, 64, p, 33, p, 4, p, 16, None) == mxq.ERR_UNSUPPORTED
    assert L.moe_dispatch(p, 0, 4, 64, 64, p, 2, None, 4, p, 16, None) == mxq.ERR_NULL
    assert L.moe_dispatch(p, 1, 4, 64, 64, p, 2, p, 4, p + 2, 16, None) == mxq.ERR_ALIGN
    assert L.moe_dispatch(None, 0, 0, 64, 64, None, 2, None, 4, None, 0, None) == mxq.OK
    assert L.moe_combine(p, 0, 16, 64, 60, p, p, 4, 2, p, None) == mxq.ERR_SHAPE
    assert L.moe_combine(p, 0, 16, 64, 64, p, p, 4, 0, p, None) == mxq.ERR_SHAPE
    assert L.moe_combine(p, 0, 16, 64, 64, None, p, 4, 2, p, None) == mxq.ERR_NULL
    assert L.moe_combine(None, 0, 0, 64, 64, None, None, 0, 2, None, None) == mxq.OK
    assert L.moe_combine_backward(p, 64, p, 64, 0, 16, 64, p, p, 4, 2, None, 4, p, p, None) == mxq.ERR_NULL
    assert L.moe_combine_backward(p, 60, p, 64, 0, 16, 64, p, p, 4, 2, p, 4, p, p, None) == mxq.ERR_SHAPE
    assert L.mxq_status_string(mxq.ERR_BAD_INDEX) == b"index out of range"


def test_workspace_sizes():
    L = mxq.lib()
    assert L.moe_dispatch_plan_workspace_bytes(2048, 64) == 0
    assert L.moe_dispatch_plan_workspace_bytes(8192, 64) == 0
    assert L.moe_dispatch_plan_workspace_bytes(8193, 64) == 5 * 64 * 4
    assert L.moe_dispatch_plan_workspace_bytes(128 * 2048 + 1, 64) == 65 * 64 * 4
    assert L.moe_route_workspace_bytes(-1, 64) == 0 and L.moe_route_workspace_bytes(16, 2000) == 0


def test_cpu_tensors_are_refused():
    x = torch.zeros(4, 8)
    ids = torch.zeros(4, 2, dtype=torch.int32)
    for call in (lambda: autograd.moe_route(x, 2), lambda: autograd.moe_dispatch(x, ids, 4),
                 lambda: autograd.moe_combine(x, ids, x, ids[0]), lambda: mxq.moe_route(x, 2), lambda: mxq.moe_dispatch_plan(ids, 4),
                 lambda: mxq.moe_dispatch(x, ids, ids[0]), lambda: mxq.moe_combine(x, ids),
                 lambda: mxq.moe_combine_backward(x, x, ids, None, ids[0])):
        with pytest.raises(TypeError):
            call()


def test_fake_shapes():
    import mxfp8_quantization_moe_device_b200.ops  # noqa: F401
    o = torch.ops.mxq
    x = torch.empty(30, 24, dtype=torch.bfloat16, device="meta")
    w, ids, counts, loss, lg = o.moe_route(x, 3, None, True)
    assert w.shape == ids.shape == (30, 3) and counts.shape == lg.shape == (24,) and loss.shape == ()
    assert w.dtype == torch.float32 and ids.dtype == counts.dtype == torch.int32
    d = o.moe_route_backward(x, w, ids, lg, w, loss, None, True)
    assert d.shape == x.shape and d.dtype == x.dtype
    pos, offs = o.moe_dispatch_plan(ids, 24)
    assert pos.shape == (30, 3) and offs.shape == (24,) and offs.dtype == torch.int32
    xs = o.moe_dispatch(x, pos, offs)
    assert xs.shape == (96, 24) and xs.dtype == x.dtype
    assert o.moe_combine(xs, pos, w).shape == (30, 24)
    dy, dw = o.moe_combine_backward(x, xs, pos, w, offs)
    assert dy.shape == (96, 24) and dw.shape == (30, 3) and dw.dtype == torch.float32


def test_overlap_of_an_output_with_strided_rows():
    """Every placement of a contiguous output against rows in a wider buffer,
    by the sets of their bytes."""
    overlaps = mxq.torch_ops().overlaps
    buf = torch.zeros(64, dtype=torch.bfloat16)
    for rows, cols, stride in ((1, 5, 9), (3, 4, 4), (3, 4, 9), (4, 1, 6), (5, 3, 7)):
        t = buf.as_strided((rows, cols), (stride, 1), 8)
        mine = {8 + i * stride + j for i in range(rows) for j in range(cols)}
        for n in (0, 1, 2, 5, 20):
            for at in range(64 - n):
                assert overlaps(buf[at:at + n], t) == bool(mine & set(range(at, at + n))), (rows, cols, stride, n, at)
    assert not overlaps(buf, buf.as_strided((0, 4), (9, 1), 8))
    # other types over the same memory
    words = buf.view(torch.int32)
    assert overlaps(words[2:5], buf[9:10]) and not overlaps(words[2:5], buf[10:12])
    assert overlaps(buf[5:7], words[3:4]) and not overlaps(buf[4:6], words[3:4])


def test_torch_module_is_rebuilt_for_another_torch(tmp_path, monkeypatch):
    from mxfp8_quantization_moe_device_b200 import build
    so = tmp_path / "_torch_ops.so"
    monkeypatch.setattr(build, "TORCH_OPS", str(so))
    monkeypatch.setattr(build, "TORCH_OPS_KEY", str(so) + ".key")
    runs = []

    def compiler(cmd, check):
        runs.append(cmd)
        with open(cmd[cmd.index("-o") + 1], "w"):
            pass

    monkeypatch.setattr(build.subprocess, "run", compiler)
    for _ in range(2):
        assert build.build_torch_ops() == str(so)
    assert len(runs) == 1 and so.exists()
    with monkeypatch.context() as m:
        m.setattr(torch, "__version__", "9.9.9")
        for _ in range(2):
            build.build_torch_ops()
        assert len(runs) == 2
    build.build_torch_ops()  # and back
    assert len(runs) == 3
    with monkeypatch.context() as m:
        m.setattr(build.sysconfig, "get_config_var", lambda name: "cpython-399")
        build.build_torch_ops()
        assert len(runs) == 4
    build.build_torch_ops()
    (tmp_path / "_torch_ops.so.key").unlink()  # built before there was a key
    build.build_torch_ops()
    assert len(runs) == 6
    build.build_torch_ops(force=True)
    assert len(runs) == 7


@pytest.mark.parametrize("there", [True, False])
def test_what_is_wrong_with_the_torch_module_is_said(there, tmp_path, monkeypatch):
    import sys
    import mxfp8_quantization_moe_device_b200 as package
    mxq.torch_ops()
    name = package.__name__ + "._torch_ops"
    monkeypatch.setattr(mxq, "_ops", None)
    monkeypatch.delattr(package, "_torch_ops")
    monkeypatch.setitem(sys.modules, name, None)  # an import that fails, with a text of its own
    if not there:
        monkeypatch.setattr(mxq, "_HERE", str(tmp_path))
    with pytest.raises(RuntimeError) as e:
        mxq.torch_ops()
    assert isinstance(e.value.__cause__, ImportError)
    assert ("is not built" in str(e.value)) == (not there) and (str(e.value.__cause__) in str(e.value)) == there
    assert "mxfp8_quantization_moe_device_b200.build" in str(e.value)


@pytest.mark.gpu
def test_registered_ops():
    import mxfp8_quantization_moe_device_b200.ops  # noqa: F401
    o = torch.ops.mxq
    x = torch.randn(30, 24, device=DEV).bfloat16()
    valid = torch.ones(30, dtype=torch.bool, device=DEV)
    w, ids, counts, loss, lg = o.moe_route(x, 3, valid, True)
    pos, offs = o.moe_dispatch_plan(ids, 24)
    xs = o.moe_dispatch(x, pos, offs)
    g = torch.ones((), device=DEV)
    for a, b in zip((w, ids, counts, loss), mxq.moe_route(x, 3, renormalize=True)):
        assert torch.equal(a, b)
    for op, args in ((o.moe_route, (x, 3, valid, True)), (o.moe_route, (x, 2, None, False)),
                     (o.moe_route_backward, (x, w, ids, lg, w, g, valid, True)), (o.moe_dispatch_plan, (ids, 24)),
                     (o.moe_dispatch, (x, pos, offs)), (o.moe_combine, (xs, pos, w)),
                     (o.moe_combine_backward, (x, xs, pos, w, offs))):
        torch.library.opcheck(op, args, test_utils=("test_schema", "test_faketensor"))


# ------------------------------------------------------------ router
ROUTE = [(1, 1, 1), (1, 4, 4), (3, 7, 2), (33, 8, 3), (40, 16, 1), (65, 24, 5), (130, 60, 4), (70, 64, 8),
         (257, 100, 6), (64, 128, 32), (300, 256, 8), (50, 257, 3), (41, 512, 10), (9, 700, 32), (21, 1024, 16)]


@pytest.mark.gpu
@pytest.mark.parametrize("T,E,k", ROUTE)
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("renorm", [False, True])
def test_route_and_gradient(T, E, k, dtype, renorm):
    l = logits_of(T, E, dtype, T + E, closed=1 if E > 4 else 0, ties=T % 2 == 0)
    g = torch.Generator().manual_seed(7)
    valid = (torch.rand(T, generator=g) < 0.8) if T > 2 else None
    gw, gl = torch.randn(T, k, generator=g), torch.tensor(3.0)
    w, ids, counts, loss, d, mag = ref_route(l, k, valid, renorm, gw, gl)
    x = l.to(DEV).requires_grad_(True)
    v = valid.to(DEV) if valid is not None else None
    gotw, goti, gotc, gotl = autograd.moe_route(x, k, valid=v, renormalize=renorm)
    assert torch.equal(goti.cpu(), ids) and torch.equal(gotc.cpu(), counts)
    near(gotw, w, 2.0 ** -18 * w + 1e-12, "weights")
    near(gotl, loss, 2.0 ** -18 * float(loss) + 1e-30, "loss")
    (gd,) = torch.autograd.grad((gotw, gotl), (x,), (gw.to(DEV), gl.to(DEV)))
    assert gd.dtype == dtype
    near(gd, d, U[dtype] * d.abs() + 2.0 ** -17 * mag + 1e-12, "gradient")
    # each gradient alone, and the forward without autograd
    only = ref_route(l, k, valid, renorm, gw, None)
    (gd,) = torch.autograd.grad(autograd.moe_route(x, k, valid=v, renormalize=renorm)[0], x, gw.to(DEV))
    near(gd, only[4], U[dtype] * only[4].abs() + 2.0 ** -17 * only[5] + 1e-12, "gradient of the weights")
    only = ref_route(l, k, valid, renorm, None, gl)
    (gd,) = torch.autograd.grad(autograd.moe_route(x, k, valid=v, renormalize=renorm)[3], x, gl.to(DEV))
    near(gd, only[4], U[dtype] * only[4].abs() + 2.0 ** -17 * only[5] + 1e-12, "gradient of the loss")
    again = mxq.moe_route(x.detach(), k, valid=v, renormalize=renorm)
    for a, b in zip(again, (gotw, goti, gotc, gotl)):
        assert torch.equal(a, b.detach())
    assert mxq.device_status() == 0


@pytest.mark.gpu
def test_route_gradient_against_differences():
    # central differences in 64 bits of the definition's value, h = 1e-5: the
    # quotient's own error is below 1e-8
    T, E, k, h = 5, 12, 3, 1e-5
    l = logits_of(T, E, torch.float32, 3)
    g = torch.Generator().manual_seed(1)
    gw = torch.randn(T, k, generator=g, dtype=torch.float64)

    def value(x):
        w, _, _, loss = ref_route(x, k, None, True)
        return float((w * gw).sum() + 2.0 * loss)

    x = l.to(DEV).requires_grad_(True)
    w, _, _, loss = autograd.moe_route(x, k, renormalize=True)
    (d,) = torch.autograd.grad((w, loss), x, (gw.float().to(DEV), torch.tensor(2.0, device=DEV)))
    for t in range(T):
        for e in range(E):
            up, dn = l.double(), l.double()
            up[t, e] += h
            dn[t, e] -= h
            num = (value(up) - value(dn)) / (2 * h)
            assert abs(num - float(d[t, e])) <= 1e-5 * (1.0 + abs(num))


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_route_rows_that_choose_nothing(dtype):
    T, E, k = 40, 20, 4
    l = logits_of(T, E, dtype, 11)
    l[0] = -math.inf                       # no expert left
    l[1] = torch.finfo(dtype).min          # the type's lowest value: choosable
    l[2, 2:] = -math.inf                   # fewer experts than slots
    l[3] = torch.finfo(dtype).max
    l[4, 1:] = torch.finfo(dtype).min
    l[12] = l[12] * 0.1 + 3e6              # far from zero, near each other
    l[13] = l[13] - 1e30
    l[14, 3] = 2e38
    valid = torch.ones(T, dtype=torch.bool)
    valid[5:9] = False
    l[6] = math.nan                        # in a padded row: not looked at
    l[7] = math.inf
    gw = torch.ones(T, k)
    w, ids, counts, loss, d, mag = ref_route(l, k, valid, True, gw, torch.tensor(1.0))
    x = l.to(DEV).requires_grad_(True)
    gotw, goti, gotc, gotl = autograd.moe_route(x, k, valid=valid.to(DEV), renormalize=True)
    assert torch.equal(goti.cpu(), ids) and torch.equal(gotc.cpu(), counts)
    near(gotw, w, 2.0 ** -18 * w + 1e-12, "weights")
    near(gotl, loss, 2.0 ** -18 * float(loss), "loss")
    (gd,) = torch.autograd.grad((gotw, gotl), x, (gw.to(DEV), torch.tensor(1.0, device=DEV)))
    near(gd, d, U[dtype] * d.abs() + 2.0 ** -17 * mag + 1e-12, "gradient")
    # a NaN or +inf in a row that counts shows in its weights and in the loss
    l[10, 3] = math.nan
    l[11, 4] = math.inf
    w, ids, counts, loss, d, mag = ref_route(l, k, valid, False, gw, torch.tensor(1.0))
    x = l.to(DEV).requires_grad_(True)
    gotw, goti, gotc, gotl = autograd.moe_route(x, k, valid=valid.to(DEV))
    assert torch.equal(goti.cpu(), ids) and torch.equal(gotc.cpu(), counts) and bool(gotl.isnan())
    near(gotw, w, 2.0 ** -18 * w.nan_to_num() + 1e-12, "weights")
    (gd,) = torch.autograd.grad(gotw, x, gw.to(DEV))
    assert bool(gd[10].isnan().all()) and bool(gd[11].isnan().all()) and not bool(gd[12:].isnan().any())
    # all tokens padded
    out = mxq.moe_route(x.detach(), k, valid=torch.zeros(T, dtype=torch.bool, device=DEV))
    assert float(out[3]) == 0.0 and int(out[2].sum()) == 0 and bool((out[1] == -1).all())


@pytest.mark.gpu
def test_route_no_tokens_strides_and_many_tokens():
    out = mxq.moe_route(torch.zeros(0, 8, device=DEV), 2)
    assert out[0].shape == (0, 2) and float(out[3]) == 0.0 and int(out[2].abs().sum()) == 0
    # rows inside a wider buffer, an odd first element
    buf = torch.randn(3000, 70, device=DEV).bfloat16()
    for view in (buf[:, :64], buf[:, 3:67], buf[::2, 1:61]):
        a, b = mxq.moe_route(view, 4, renormalize=True), mxq.moe_route(view.contiguous(), 4, renormalize=True)
        for p, q in zip(a, b):
            assert torch.equal(p, q)
    # more tokens than the grid takes at once: against torch in 64 bits
    T, E, k = 70001, 64, 6
    l = torch.randn(T, E, device=DEV)
    w, ids, counts, loss = mxq.moe_route(l, k)
    p = torch.softmax(l.double(), 1)
    ri = torch.sort(l, dim=1, descending=True, stable=True).indices[:, :k]
    assert torch.equal(ids.long(), ri)
    rc = torch.bincount(ri.reshape(-1), minlength=E)
    assert torch.equal(counts.long(), rc)
    rl = E * float((rc.double() / (k * T) * p.mean(0)).sum())
    assert abs(float(loss) - rl) <= 2.0 ** -18 * rl
    near(w, p.gather(1, ri).cpu(), 2.0 ** -18 * p.gather(1, ri).cpu(), "weights")
    for _ in range(3):
        again = mxq.moe_route(l, k)
        assert all(torch.equal(a, b) for a, b in zip(again, (w, ids, counts, loss)))


# ------------------------------------------------------------ order by expert
@pytest.mark.gpu
@pytest.mark.parametrize("T,E,k", [(0, 5, 2), (1, 1, 1), (5, 3, 2), (100, 16, 4), (1024, 60, 8), (1025, 64, 8),
                                   (3000, 7, 6), (2000, 1024, 32), (300, 1000, 5), (4096, 4, 4), (4000, 3, 2),
                                   (8193, 33, 1), (8192, 1, 1)])
@pytest.mark.parametrize("dropped", [0.0, 0.3])
def test_plan(T, E, k, dropped):
    ids = ids_of(T, E, k, T + E + k, dropped)
    pos, offs = mxq.moe_dispatch_plan(ids.to(DEV), E)
    rp, ro = ref_plan(ids, E)
    assert torch.equal(pos.cpu(), rp) and torch.equal(offs.cpu(), ro)
    assert mxq.device_status() == 0


@pytest.mark.gpu
def test_plan_many_entries_one_expert_and_bad_ids():
    # several tiles per chunk, against a stable sort
    T, E, k = 90001, 37, 8
    ids = torch.randint(0, E, (T, k), device=DEV, dtype=torch.int32)
    ids[torch.rand(T, k, device=DEV) < 0.1] = -1
    for x in (ids, torch.full_like(ids, 36), torch.full_like(ids, -5)):
        pos, offs = mxq.moe_dispatch_plan(x, E)
        flat = x.reshape(-1).long()
        key = torch.where(flat < 0, E, flat)
        order = torch.sort(key, stable=True).indices
        want = torch.empty_like(flat)
        want[order] = torch.arange(flat.numel(), device=DEV)
        want[flat < 0] = -1
        assert torch.equal(pos.reshape(-1).long(), want)
        assert torch.equal(offs.long(), torch.cumsum(torch.bincount(key, minlength=E + 1)[:E], 0))
    # the same expert twice in a token: two rows, the first slot first
    pos, offs = mxq.moe_dispatch_plan(torch.tensor([[2, 2], [0, 2]], dtype=torch.int32, device=DEV), 3)
    assert pos.tolist() == [[1, 2], [0, 3]] and offs.tolist() == [1, 1, 4]
    # an id past the experts is dropped and reported
    pos, offs = mxq.moe_dispatch_plan(torch.tensor([[3, 1], [0, 9]], dtype=torch.int32, device=DEV), 3)
    assert pos.tolist() == [[-1, 1], [0, -1]] and offs.tolist() == [1, 2, 2]
    assert mxq.device_status() == mxq.ERR_BAD_INDEX and mxq.device_status() == 0


# ------------------------------------------------------------ rows
ROWS = [(0, 4, 2, 64), (1, 3, 1, 1), (3, 4, 2, 8), (17, 5, 3, 63), (50, 16, 2, 2048), (33, 60, 6, 1419),
        (129, 8, 8, 514), (20, 40, 32, 100), (7, 4, 2, 7168), (260, 4, 4, 130), (11, 6, 5, 31), (40, 12, 5, 37), (6, 3, 2, 33)]


@pytest.mark.gpu
@pytest.mark.parametrize("T,E,k,K", ROWS)
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("dropped", [0.0, 0.25, 1.0])
def test_dispatch_combine_and_gradients(T, E, k, K, dtype, dropped):
    g = torch.Generator().manual_seed(T + K)
    ids = ids_of(T, E, k, 5 * T + k, dropped)
    x = torch.randn(T, K, generator=g).to(dtype)
    w = torch.randn(T, k, generator=g)
    xd, wd = x.to(DEV).requires_grad_(True), w.to(DEV).requires_grad_(True)
    xs, pos, offs = autograd.moe_dispatch(xd, ids.to(DEV), E)
    M = mxq.moe_dispatch_rows(T * k)
    rp, ro = ref_plan(ids, E)
    assert torch.equal(pos.cpu(), rp) and torch.equal(offs.cpu(), ro) and xs.shape == (M, K)
    want = torch.zeros(M, K, dtype=dtype)
    for t in range(T):
        for j in range(k):
            if rp[t, j] >= 0:
                want[rp[t, j]] = x[t]
    assert torch.equal(xs.detach().cpu(), want)
    gxs = torch.randn(M, K, generator=g).to(dtype)
    (dx,) = torch.autograd.grad(xs, xd, gxs.to(DEV))
    live = (rp >= 0)[..., None].double()
    rows = gxs.double()[rp.clamp(min=0).long().reshape(-1)].reshape(T, k, K) * live if M else torch.zeros(T, k, K)
    ref, mag = rows.sum(1), rows.abs().sum(1)
    near(dx, ref, U[dtype] * ref.abs() + (k + 1) * 2.0 ** -24 * mag, "gradient of dispatch")
    # combine
    y = torch.randn(M, K, generator=g).to(dtype)
    yd = y.to(DEV).requires_grad_(True)
    out = autograd.moe_combine(yd, pos, wd, offs)
    rows = y.double()[rp.clamp(min=0).long().reshape(-1)].reshape(T, k, K) if M else torch.zeros(T, k, K)
    terms = rows * w.double()[..., None] * live
    near(out, terms.sum(1), U[dtype] * terms.sum(1).abs() + (k + 1) * 2.0 ** -24 * terms.abs().sum(1), "combine")
    dout = torch.randn(T, K, generator=g).to(dtype)
    dy, dw = torch.autograd.grad(out, (yd, wd), dout.to(DEV))
    ref = torch.zeros(M, K, dtype=torch.float64)
    for t in range(T):
        for j in range(k):
            if rp[t, j] >= 0:
                ref[rp[t, j]] = w[t, j].double() * dout[t].double()
    near(dy, ref, U[dtype] * ref.abs() + 2.0 ** -24 * ref.abs(), "gradient of combine by rows")
    dots = rows * dout.double()[:, None, :] * live
    near(dw, dots.sum(2), (K + 1) * 2.0 ** -24 * dots.abs().sum(2), "gradient of combine by weights")
    # no weights: ones
    ones = mxq.moe_combine(yd.detach(), pos)
    assert torch.equal(ones, mxq.moe_combine(yd.detach(), pos, torch.ones(T, k, device=DEV)))
    assert mxq.device_status() == 0


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_rows_strides_offsets_and_poison(dtype):
    T, E, k = 37, 6, 3
    ids = ids_of(T, E, k, 1, 0.2).to(DEV)
    pos, offs = mxq.moe_dispatch_plan(ids, E)
    M, n = mxq.moe_dispatch_rows(T * k), int(offs[-1])
    w = torch.rand(T, k, device=DEV)
    buf = torch.randn(T, 300, device=DEV).to(dtype)
    for lo, hi in ((0, 256), (8, 264), (2, 258), (1, 258), (4, 260)):
        v = buf[:, lo:hi]
        xs = mxq.moe_dispatch(v, pos, offs)
        assert torch.equal(xs, mxq.moe_dispatch(v.contiguous(), pos, offs))
        wide = torch.full((M, 300), math.nan, device=DEV).to(dtype)
        wide[:, lo:hi] = xs
        y = wide[:, lo:hi]
        y[n:] = math.nan  # rows behind the last group are not read
        assert torch.equal(mxq.moe_combine(y, pos, w), mxq.moe_combine(y.contiguous(), pos, w))
        assert not bool(mxq.moe_combine(y, pos, w).isnan().any())
        a = mxq.moe_combine_backward(v, y, pos, w, offs)
        b = mxq.moe_combine_backward(v.contiguous(), y.contiguous(), pos, w, offs)
        assert torch.equal(a[0], b[0])
        # rows on other boundaries move in other vectors, so a dot's terms are
        # added in another order: two sums of K terms, each within K 2^-24 of
        # the sum of absolute values
        K = hi - lo
        mag = (v.double().abs() @ torch.nan_to_num(y.double()).abs().t()).gather(1, pos.clamp(min=0).long())
        near(a[1], b[1].cpu(), 2 * K * 2.0 ** -24 * mag.cpu(), "dots of strided rows")
        assert bool((a[0][n:] == 0).all()) and not bool(a[1].isnan().any())
        only_y = mxq.moe_combine_backward(v, y, pos, w, offs, need_weights=False)
        only_w = mxq.moe_combine_backward(v, y, pos, w, offs, need_y=False)
        assert only_y[1] is None and only_w[0] is None
        assert torch.equal(only_y[0], a[0]) and torch.equal(only_w[1], a[1])
    # a place past the rows is skipped and reported; fewer rows than places
    short = mxq.moe_dispatch(buf, pos, offs, out=torch.empty(16, 300, dtype=dtype, device=DEV))
    assert torch.equal(short, mxq.moe_dispatch(buf, pos, offs)[:16]) and mxq.device_status() == mxq.ERR_BAD_INDEX
    mxq.moe_combine(torch.zeros(16, 300, dtype=dtype, device=DEV), pos, w)
    assert mxq.device_status() == mxq.ERR_BAD_INDEX and mxq.device_status() == 0


@pytest.mark.gpu
def test_more_than_2_31_elements():
    # dispatched rows and logits whose last elements lie behind 2^31
    T, E, k, K = 66000, 12, 8, 4096
    ids = torch.stack([torch.randperm(E, device=DEV)[:k] for _ in range(50)]).repeat(T // 50, 1).to(torch.int32)
    ids[-7:, 3] = -1
    x = torch.randn(T, K, device=DEV).bfloat16()
    pos, offs = mxq.moe_dispatch_plan(ids, E)
    xs = mxq.moe_dispatch(x, pos, offs)
    assert xs.numel() > 2 ** 31 and int(offs[-1]) == T * k - 7
    assert bool((xs[int(offs[-1]):] == 0).all())
    top = torch.argsort(pos.reshape(-1))[-3000:]  # the entries of the last rows
    assert torch.equal(xs[pos.reshape(-1)[top].long()], x[top // k])
    w = torch.full((T, k), 0.25, device=DEV)
    got = mxq.moe_combine(xs, pos, w)  # eight equal rows at a quarter: exact
    assert torch.equal(got[:-7], (2 * x[:-7].float()).bfloat16())
    dy, dw = mxq.moe_combine_backward(x, xs, pos, w, offs)
    assert torch.equal(dy[pos.reshape(-1)[top].long()], (0.25 * x[top // k].float()).bfloat16())
    sq = x.double().square().sum(1)
    assert bool(((dw[:-7].double() - sq[:-7, None]).abs() <= K * 2.0 ** -24 * sq[:-7, None]).all())
    del xs, dy
    T, E = 2100000, 1024
    l = torch.randn(T, E, device=DEV, dtype=torch.bfloat16)
    w, ids, counts, loss = mxq.moe_route(l, 2)
    assert l.numel() > 2 ** 31 and int(counts.sum()) == 2 * T
    tail = l[-1000:]
    ri = torch.sort(tail.float(), dim=1, descending=True, stable=True).indices[:, :2]
    p = torch.softmax(tail.double(), 1).gather(1, ri)
    assert torch.equal(ids[-1000:].long(), ri)
    near(w[-1000:], p.cpu(), 2.0 ** -18 * p.cpu(), "weights")
    assert mxq.device_status() == 0


@pytest.mark.gpu
def test_refusals_of_the_binding():
    x = torch.randn(8, 64, device=DEV).bfloat16()
    ids = torch.zeros(8, 2, dtype=torch.int32, device=DEV)
    pos, offs = mxq.moe_dispatch_plan(ids, 4)
    w = torch.ones(8, 2, device=DEV)
    bad = [lambda: mxq.moe_route(x.half(), 2), lambda: mxq.moe_route(x.t(), 2), lambda: mxq.moe_route(x[0], 2),
           lambda: mxq.moe_route(x[:1].expand(8, 64), 2), lambda: mxq.moe_route(x, 2, valid=w[:, 0]),
           lambda: mxq.moe_route(x, 2, valid=torch.ones(7, dtype=torch.bool, device=DEV)),
           lambda: mxq.moe_route(x, 2, ids=ids.long()), lambda: mxq.moe_dispatch_plan(ids.long(), 4),
           lambda: mxq.moe_dispatch_plan(ids.t(), 4), lambda: mxq.moe_dispatch(x, pos[:7], offs),
           lambda: mxq.moe_dispatch(x, pos, offs.long()), lambda: mxq.moe_dispatch(x.t(), pos, offs),
           lambda: mxq.moe_dispatch(x, pos, offs, out=torch.empty(16, 63, device=DEV).bfloat16()),
           lambda: mxq.moe_combine(x, pos, w.double()), lambda: mxq.moe_combine(x, pos, w[:, :1]),
           lambda: mxq.moe_combine(x, pos.long(), w), lambda: mxq.moe_combine_backward(x.float(), x, pos, w, offs),
           lambda: mxq.moe_combine_backward(x[:, :32], x, pos, w, offs),
           lambda: mxq.moe_route_backward(x, w, ids.long(), None, w, None),
           lambda: mxq.moe_route_backward(x, w, ids, None, w, w[0, 0])]
    for call in bad:
        with pytest.raises(TypeError):
            call()
    for call in (lambda: mxq.moe_route(x, 0), lambda: mxq.moe_route(x, 65), lambda: mxq.moe_dispatch_plan(ids, 0),
                 lambda: mxq.moe_combine(x, pos[:, :0])):
        with pytest.raises(ValueError):
            call()
    with pytest.raises(mxq.MXQError):
        mxq.moe_route(x, 33)
    assert mxq.device_status() == 0


@pytest.mark.gpu
def test_refusals_of_the_differentiable_calls():
    x = torch.randn(8, 64, device=DEV).bfloat16()
    ids = torch.zeros(8, 2, dtype=torch.int32, device=DEV)
    xs, pos, offs = autograd.moe_dispatch(x, ids, 4)
    w = torch.ones(8, 2, device=DEV)
    for call in (lambda: autograd.moe_route(x.half(), 2), lambda: autograd.moe_route(x.t(), 2),
                 lambda: autograd.moe_route(x[:1].expand(8, 64), 2), lambda: autograd.moe_route(x, 2, valid=w[:, 0]),
                 lambda: autograd.moe_dispatch(x, ids.long(), 4), lambda: autograd.moe_dispatch(x, ids[:7], 4),
                 lambda: autograd.moe_dispatch(x.t(), ids, 4), lambda: autograd.moe_combine(xs, pos, w.double(), offs),
                 lambda: autograd.moe_combine(xs, pos.long(), w, offs),
                 lambda: autograd.moe_combine(xs, pos, w, offs.cpu())):
        with pytest.raises(TypeError):
            call()
    for call in (lambda: autograd.moe_route(x, 0), lambda: autograd.moe_route(x, 65),
                 lambda: autograd.moe_dispatch(x, ids, 0)):
        with pytest.raises(ValueError):
            call()
    with pytest.raises(mxq.MXQError) as e:
        autograd.moe_route(x, 33)
    assert e.value.code == mxq.ERR_UNSUPPORTED
    assert mxq.device_status() == 0


@pytest.mark.gpu
def test_gradients_through_odd_incoming_gradients():
    """Expanded, strided and missing incoming gradients, a leaf that wants
    none, and a second differentiation, which is refused."""
    T, E, k, K = 30, 8, 2, 40
    l = torch.randn(T, E, device=DEV, requires_grad=True)
    x = torch.randn(T, K, device=DEV, requires_grad=True)
    w, ids, counts, loss = autograd.moe_route(l, k)
    assert not ids.requires_grad and not counts.requires_grad and w.requires_grad and loss.requires_grad
    xs, pos, offs = autograd.moe_dispatch(x, ids, E)
    y = autograd.moe_combine(xs, pos, w, offs)
    gl, gx = torch.autograd.grad(y.sum() + 2 * loss, (l, x), retain_graph=True)  # a gradient of expanded ones
    rl, rx = torch.autograd.grad((y, loss), (l, x), (torch.ones_like(y), torch.tensor(2.0, device=DEV)),
                                 retain_graph=True)
    assert torch.equal(gl, rl) and torch.equal(gx, rx)
    g = torch.randn(K, T, device=DEV).t()
    a = torch.autograd.grad(y, (l, x), g, retain_graph=True)
    b = torch.autograd.grad(y, (l, x), g.contiguous(), retain_graph=True)
    assert all(torch.equal(p, q) for p, q in zip(a, b))
    assert torch.autograd.grad(y, (l,), g, retain_graph=True)[0].shape == l.shape
    const = autograd.moe_combine(xs.detach(), pos, w.detach(), offs)
    assert not const.requires_grad
    only = autograd.moe_combine(xs.detach(), pos, w, offs)
    torch.autograd.grad(only.sum(), (l,), retain_graph=True)
    (first,) = torch.autograd.grad(y.sum(), (x,), create_graph=True)
    with pytest.raises(RuntimeError, match="differentiated again"):
        first.sum().backward(retain_graph=True)
    with pytest.raises(RuntimeError):  # the graph ends there, as with torch's once_differentiable
        torch.autograd.grad(first.sum(), (x,))
    (first,) = torch.autograd.grad(loss, (l,), create_graph=True)
    with pytest.raises(RuntimeError, match="differentiated again"):
        first.square().sum().backward()
    assert mxq.device_status() == 0


# ------------------------------------------------------------ together
def _layer(x, wr, we, k, offs_check=None):
    logits = x @ wr
    w, ids, counts, loss = autograd.moe_route(logits, k, renormalize=True)
    xs, pos, offs = autograd.moe_dispatch(x, ids, we.shape[0])
    y = autograd.fp8_grouped_mm(xs, we, offs)
    return autograd.moe_combine(y, pos, w, offs), counts, offs, loss


@pytest.mark.gpu
def test_layer_forward_and_backward():
    """Router, dispatch, the FP8 grouped product and combine as one layer,
    against the same layer with exact products: an e4m3 operand is off by up
    to 2^-4 of its value, about 0.026 in the mean square, so a product of two
    is off by about 0.037 of its norm, and a gradient by the router on top of
    it stays below 0.08 (the bound of the grouped product's own tests)."""
    T, E, k, K, N = 200, 6, 2, 256, 128
    g = torch.Generator(device=DEV).manual_seed(3)
    x = torch.randn(T, K, generator=g, device=DEV).bfloat16().requires_grad_(True)
    wr = (torch.randn(K, E, generator=g, device=DEV) * 0.1).bfloat16().requires_grad_(True)
    we = (torch.randn(E, N, K, generator=g, device=DEV) * 0.05).bfloat16().requires_grad_(True)
    dout = torch.randn(T, N, generator=g, device=DEV).bfloat16()
    out, counts, offs, loss = _layer(x, wr, we, k)
    assert torch.equal(torch.cumsum(counts, 0).int(), offs)
    grads = torch.autograd.grad((out, loss), (x, wr, we), (dout, torch.tensor(0.5, device=DEV)))
    # the same in 64 bits with the logits' bf16 rounding kept
    xr, wrr, wer = (t.detach().double().requires_grad_(True) for t in (x, wr, we))
    lg = xr @ wrr
    lg = lg + ((x.detach() @ wr.detach()).double() - lg).detach()
    p = torch.softmax(lg, 1)
    ids = torch.sort(lg.detach(), dim=1, descending=True, stable=True).indices[:, :k]
    w = p.gather(1, ids)
    w = w / w.sum(1, keepdim=True)
    ref = sum(w[:, j:j + 1] * torch.einsum("tk,tnk->tn", xr, wer[ids[:, j]]) for j in range(k))
    f = torch.bincount(ids.reshape(-1), minlength=E).double() / (k * T)
    rl = E * (f * p.mean(0)).sum()
    want = torch.autograd.grad((ref, rl), (xr, wrr, wer), (dout.double(), torch.tensor(0.5, device=DEV).double()))
    assert abs(float(loss.detach()) - float(rl.detach())) <= 2.0 ** -17 * float(rl.detach())
    for got, r, name in zip((out, *grads), (ref, *want), ("out", "dx", "dwr", "dwe")):
        assert torch.linalg.norm(got.detach().double() - r.detach()) <= 0.08 * torch.linalg.norm(r.detach()), name
    assert mxq.device_status() == 0


@pytest.mark.gpu
def test_streams_graphs_and_calls_at_once():
    T, E, k, K = 20000, 64, 4, 256
    l = torch.randn(T, E, device=DEV).bfloat16()
    x = torch.randn(T, K, device=DEV).bfloat16()

    def step():
        w, ids, counts, loss = mxq.moe_route(l, k, renormalize=True)
        pos, offs = mxq.moe_dispatch_plan(ids, E)
        xs = mxq.moe_dispatch(x, pos, offs)
        return [w, ids, counts, loss, pos, offs, xs, mxq.moe_combine(xs, pos, w),
                *mxq.moe_combine_backward(x, xs, pos, w, offs)]

    want = step()
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(3)]
    got = []
    for s in streams:
        s.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(s):
            got.append(step())
    torch.cuda.synchronize()
    for r in got:
        assert all(torch.equal(a, b) for a, b in zip(r, want))
    # two graphs of the same step on new inputs, replayed at once on two streams
    graphs = []
    for _ in range(2):
        gr = torch.cuda.CUDAGraph()
        with torch.cuda.graph(gr):
            graphs.append((gr, step()))
    l.copy_(torch.randn(T, E, device=DEV))
    x.copy_(torch.randn(T, K, device=DEV))
    torch.cuda.synchronize()
    for (gr, _), s in zip([g for g in graphs], streams):
        with torch.cuda.stream(s):
            gr.replay()
    torch.cuda.synchronize()
    want = step()
    torch.cuda.synchronize()
    for _, out in graphs:
        assert all(torch.equal(a, b) for a, b in zip(out, want))
    assert mxq.device_status() == 0


def _train(l, x, k):
    """a step of router, dispatch and combine through the differentiable calls"""
    w, ids, counts, loss = autograd.moe_route(l, k, renormalize=True)
    xs, pos, offs = autograd.moe_dispatch(x, ids, l.shape[1])
    out = autograd.moe_combine(xs, pos, w, offs)
    return torch.autograd.grad((out, loss), (l, x), (x.detach(), torch.ones_like(loss)))


@pytest.mark.gpu
def test_captured_training_step():
    T, E, k, K = 777, 24, 3, 200
    l = torch.randn(T, E, device=DEV).bfloat16().requires_grad_(True)
    x = torch.randn(T, K, device=DEV).bfloat16().requires_grad_(True)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        _train(l, x, k)
    torch.cuda.current_stream().wait_stream(side)
    gr = torch.cuda.CUDAGraph()
    with torch.cuda.graph(gr):
        got = _train(l, x, k)
    with torch.no_grad():
        l.copy_(torch.randn(T, E, device=DEV))
        x.copy_(torch.randn(T, K, device=DEV))
    gr.replay()
    gr.replay()
    torch.cuda.synchronize()
    want = _train(l, x, k)
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    assert mxq.device_status() == 0


@pytest.mark.gpu
def test_capture_beside_a_living_graph_is_refused():
    T, E, k, K = 64, 8, 2, 64
    l = torch.randn(T, E, device=DEV).requires_grad_(True)
    x = torch.randn(T, K, device=DEV).requires_grad_(True)
    w, ids, _, _ = autograd.moe_route(l, k)  # graphs on the default stream that live on
    xs, pos, offs = autograd.moe_dispatch(x, ids, E)
    xd, wd, ld = x.detach(), w.detach(), l.detach()
    calls = (lambda: autograd.moe_route(l, k), lambda: autograd.moe_dispatch(x, ids, E),
             lambda: autograd.moe_combine(xs, pos, wd, offs), lambda: autograd.moe_combine(xs.detach(), pos, w, offs))
    torch.cuda.synchronize()
    gr = torch.cuda.CUDAGraph()
    with torch.cuda.graph(gr):
        for call in calls:
            with pytest.raises(RuntimeError, match="default stream before this capture"):
                call()
        with torch.no_grad():
            a = autograd.moe_route(l, k)[0]
        b = autograd.moe_route(ld.requires_grad_(True), k)[0].detach()  # a leaf of its own
    gr.replay()
    torch.cuda.synchronize()
    assert torch.equal(a, w) and torch.equal(b, w) and torch.equal(mxq.moe_dispatch(xd, pos, offs), xs)


@pytest.mark.gpu
def test_outputs_over_inputs_are_refused():
    T, E, k, K = 16, 4, 1, 64
    x = torch.randn(T, K, device=DEV)
    l = torch.randn(T, E, device=DEV)
    g = torch.zeros(E, device=DEV)
    w, ids, _, _ = mxq.moe_route(l, k, loss_grad=g)
    pos, offs = mxq.moe_dispatch_plan(ids, E)
    y, big = mxq.moe_dispatch(x, pos, offs), torch.randn(2 * T, K, device=DEV)
    for call in (lambda: mxq.moe_dispatch(x, pos, offs, out=x), lambda: mxq.moe_combine(y, pos, w, out=y),
                 lambda: mxq.moe_combine(big[:T], pos, w, out=big[1:T + 1]),
                 lambda: mxq.moe_combine_backward(x, y, pos, w, offs, grad_y=y),
                 lambda: mxq.moe_combine_backward(x, y, pos, w, offs, grad_y=x),
                 lambda: mxq.moe_route_backward(l, w, ids, g, w, None, out=l)):
        with pytest.raises(ValueError, match="overlap"):
            call()
    assert torch.equal(mxq.moe_combine(big[:T], pos, w, out=big[T:]), mxq.moe_combine(big[:T].clone(), pos, w))


@pytest.mark.gpu
def test_outputs_over_strided_rows_are_refused():
    T, E, k, K = 16, 4, 1, 64
    buf = torch.randn(4 * T, 2 * K, device=DEV)
    x, y, l = buf[:T, :K], buf[T:2 * T, K:], buf[2 * T:3 * T, 8:8 + E]
    before = buf.clone()
    g = torch.zeros(E, device=DEV)
    w, ids, _, _ = mxq.moe_route(l, k, loss_grad=g)
    pos, offs = mxq.moe_dispatch_plan(ids, E)
    flat = buf.view(-1)
    over_x = flat[2 * K:2 * K + T * K].view(T, K)  # from the second row of x on
    over_y = flat[2 * K * T:2 * K * T + T * K].view(T, K)
    over_l = flat[2 * T * 2 * K + 8 + E - 1:][:T * E].view(T, E)  # the first row's last logit
    for call in (lambda: mxq.moe_dispatch(x, pos, offs, out=over_x), lambda: mxq.moe_combine(y, pos, w, out=over_y),
                 lambda: mxq.moe_combine_backward(x, y, pos, w, offs, grad_y=over_x),
                 lambda: mxq.moe_combine_backward(x, y, pos, w, offs, grad_y=over_y),
                 lambda: mxq.moe_route_backward(l, w, ids, g, w, None, out=over_l)):
        with pytest.raises(ValueError, match="overlap"):
            call()
    assert torch.equal(buf, before)
    # between two rows there is room
    gap = flat[2 * K + K:2 * K + 2 * K].view(1, K)
    row = mxq.moe_combine(x, torch.tensor([[3]], dtype=torch.int32, device=DEV), out=gap)
    assert torch.equal(row[0], x[3])
    assert mxq.device_status() == 0


@pytest.mark.gpu
@pytest.mark.parametrize("T,k", [(1, 1), (16, 2), (2048, 2), (5000, 4)])  # one tile, one launch of several, two launches
def test_places_over_their_ids_are_refused(T, k):
    E = 8
    ids = ids_of(T, E, k, T).to(DEV)
    want = mxq.moe_dispatch_plan(ids, E)
    buf = torch.zeros(2 * T * k + E, dtype=torch.int32, device=DEV)
    inside = buf[E:E + T * k].view(T, k)
    inside.copy_(ids)
    before = buf.clone()
    for call in (lambda: mxq.moe_dispatch_plan(inside, E, pos=inside), lambda: mxq.moe_dispatch_plan(inside, E, offs=buf[1:E + 1]),
                 lambda: mxq.moe_dispatch_plan(inside, E, pos=buf[E + T * k - 1:][:T * k].view(T, k)),
                 lambda: mxq.moe_dispatch_plan(ids, E, pos=inside, offs=buf[1:E + 1])):
        with pytest.raises(ValueError, match="overlap"):
            call()
    assert torch.equal(buf, before)
    # right beside one another
    got = mxq.moe_dispatch_plan(inside, E, pos=buf[E + T * k:].view(T, k), offs=buf[:E])
    assert all(torch.equal(a, b) for a, b in zip(got, want)) and torch.equal(inside, ids)
    assert mxq.device_status() == 0


@pytest.mark.gpu
def test_outputs_of_the_router_apart():
    T, E, k = 40, 8, 2
    l = torch.randn(T, E, device=DEV)
    valid = torch.ones(T, dtype=torch.bool, device=DEV)
    g = torch.zeros(E, device=DEV)
    w, ids, _, _ = mxq.moe_route(l, k, valid=valid, loss_grad=g)
    flat = l.view(-1)
    ints = flat.view(torch.int32)
    a = torch.zeros(T * k, device=DEV)
    gw, gl = torch.ones(T, k, device=DEV), torch.ones((), device=DEV)
    big = torch.zeros(4 * T * E, device=DEV)
    kept = [t.clone() for t in (l, valid, a, w, ids, g)]
    for call in (lambda: mxq.moe_route(l, k, weights=flat[T * E - T * k:].view(T, k)),
                 lambda: mxq.moe_route(l, k, ids=ints[:T * k].view(T, k)),
                 lambda: mxq.moe_route(l, k, counts=ints[5:5 + E]), lambda: mxq.moe_route(l, k, loss=flat[7]),
                 lambda: mxq.moe_route(l, k, loss_grad=flat[:E]),
                 lambda: mxq.moe_route(l, k, valid=valid, counts=valid.view(torch.int32)[2:2 + E]),
                 lambda: mxq.moe_route(l, k, weights=a.view(T, k), ids=a.view(torch.int32).view(T, k)),
                 lambda: mxq.moe_route(l, k, weights=a.view(T, k), loss=a[3]),
                 lambda: mxq.moe_route(l, k, loss=g[E - 1], loss_grad=g),
                 lambda: mxq.moe_route(l, k, counts=a[:E].view(torch.int32), loss_grad=a[E - 1:2 * E - 1])):
        with pytest.raises(ValueError, match="overlap"):
            call()
    for t, n in ((w, T * k), (gw, T * k), (ids, T * k), (g, E), (gl, 1)):
        part = big[T * E - n:T * E].view(t.dtype).view(t.shape)
        part.copy_(t)
        args = [part if t is x else x for x in (w, ids, g, gw, gl)]
        with pytest.raises(ValueError, match="overlap"):
            mxq.moe_route_backward(l, *args, out=big[:T * E].view(T, E))
        want = mxq.moe_route_backward(l, w, ids, g, gw, gl)
        assert torch.equal(mxq.moe_route_backward(l, *args, out=big[T * E:2 * T * E].view(T, E)), want)
    assert all(torch.equal(t, b) for t, b in zip((l, valid, a, w, ids, g), kept))
    # side by side in one buffer
    o = torch.zeros(2 * T * k + 2 * E + 1, device=DEV)
    i = o.view(torch.int32)
    got = mxq.moe_route(l, k, weights=o[:T * k].view(T, k), ids=i[T * k:2 * T * k].view(T, k), counts=i[2 * T * k:][:E],
                        loss=o[-1], loss_grad=o[2 * T * k + E:][:E])
    assert all(torch.equal(a, b) for a, b in zip(got, mxq.moe_route(l, k))) and torch.equal(o[-1 - E:-1], g)
    assert mxq.device_status() == 0


@pytest.mark.gpu
@pytest.mark.parametrize("T,k,K", [(16, 2, 64), (300, 3, 130)])
def test_outputs_of_the_row_movement_apart(T, k, K):
    E = 5
    x = torch.randn(T, K, device=DEV)
    w, dout = torch.rand(T, k, device=DEV), torch.randn(T, K, device=DEV)
    pos, offs = mxq.moe_dispatch_plan(ids_of(T, E, k, 3, 0.2).to(DEV), E)
    M = mxq.moe_dispatch_rows(T * k)
    y = mxq.moe_dispatch(x, pos, offs)
    out, (dy, dw) = mxq.moe_combine(y, pos, w), mxq.moe_combine_backward(dout, y, pos, w, offs)
    size = max(M * K, T * K)
    big = torch.zeros(2 * size, device=DEV)
    calls = {"dispatch": lambda p, o, ww, at: mxq.moe_dispatch(x, p, o, out=big[at:at + M * K].view(M, K)),
             "combine": lambda p, o, ww, at: mxq.moe_combine(y, p, ww, out=big[at:at + T * K].view(T, K)),
             "rows": lambda p, o, ww, at: mxq.moe_combine_backward(dout, y, p, ww, o, grad_y=big[at:at + M * K].view(M, K))[0]}
    want = {"dispatch": y, "combine": out, "rows": dy}
    reads = {"dispatch": (pos, offs), "combine": (pos, w), "rows": (pos, offs, w)}
    for name, call in calls.items():
        for t in reads[name]:
            part = big[5:5 + t.numel()].view(t.dtype).view(t.shape)
            part.copy_(t)
            args = [part if t is v else v for v in (pos, offs, w)]
            with pytest.raises(ValueError, match="overlap an input"):
                call(*args, 0)
            assert torch.equal(call(*args, size), want[name])
    # the weights' gradient over what is read, and over the rows'
    buf = torch.zeros(M * K + T * k, device=DEV)
    over = buf[M * K - 1:][:T * k].view(T, k)
    for kw in ({"grad_weights": w}, {"grad_weights": pos.view(torch.float32)}, {"grad_weights": dout.view(-1)[:T * k].view(T, k)},
               {"grad_weights": y.view(-1)[K:][:T * k].view(T, k)}, {"grad_weights": w, "need_y": False},
               {"grad_y": buf[:M * K].view(M, K), "grad_weights": over}):
        with pytest.raises(ValueError, match="overlap"):
            mxq.moe_combine_backward(dout, y, pos, w, offs, **kw)
    a = mxq.moe_combine_backward(dout, y, pos, w, offs, grad_y=buf[:M * K].view(M, K), grad_weights=buf[M * K:].view(T, k))
    assert torch.equal(a[0], dy) and torch.equal(a[1], dw)
    # what is not asked for is not looked at
    b = mxq.moe_combine_backward(dout, y, pos, w, offs, need_weights=False, grad_weights=w)
    assert torch.equal(b[0], dy) and b[1] is None
    assert mxq.device_status() == 0


@pytest.mark.gpu
def test_captured_backward_into_a_living_graph_is_refused():
    """The inputs come out of operations within the capture, the leaf behind
    them also belongs to a graph on the default stream that lives on."""
    T, E, k, K = 64, 8, 2, 64
    x = torch.randn(T, K, device=DEV)
    bias = torch.randn(E, device=DEV, requires_grad=True)
    base = torch.randn(T, E, device=DEV)
    scale = torch.ones(K, device=DEV, requires_grad=True)
    share = torch.ones((), device=DEV, requires_grad=True)
    keep = [base + bias, x * scale, share * 1.0]
    w, ids, _, _ = mxq.moe_route(keep[0].detach(), k)
    xs, pos, offs = autograd.moe_dispatch(x, ids, E)
    dl = torch.randn(T, k, device=DEV)
    dx, dout = torch.randn(xs.shape, device=DEV), torch.randn(T, K, device=DEV)
    torch.cuda.synchronize()
    gr = torch.cuda.CUDAGraph()
    with torch.cuda.graph(gr):
        logits = base + bias
        got, _, _, loss = autograd.moe_route(logits, k)
        rows = autograd.moe_dispatch(x * scale, ids, E)[0]
        out = autograd.moe_combine(xs, pos, w * share, offs)
        both = autograd.moe_combine(rows, pos, w, offs)
        for call in (lambda: torch.autograd.grad(got, bias, dl, retain_graph=True),
                     lambda: torch.autograd.grad(loss, bias, retain_graph=True),
                     lambda: got.backward(dl, retain_graph=True),
                     lambda: torch.autograd.grad(rows, scale, dx, retain_graph=True),
                     lambda: torch.autograd.grad(out, share, dout, retain_graph=True),
                     lambda: torch.autograd.grad(both, scale, dout, retain_graph=True)):
            with pytest.raises(RuntimeError, match="default stream before this capture"):
                call()
        (inner,) = torch.autograd.grad(got, logits, dl)  # ends before the leaf
    gr.replay()
    torch.cuda.synchronize()
    l = keep[0].detach().requires_grad_(True)
    assert torch.equal(got, w) and torch.equal(inner, torch.autograd.grad(autograd.moe_route(l, k)[0], l, dl)[0])
    assert bias.grad is None and torch.equal(both, mxq.moe_combine(mxq.moe_dispatch(x, pos, offs), pos, w))
    # the same with that graph gone
    del keep, logits, got, loss, rows, out, both, call
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        torch.autograd.grad(autograd.moe_route(base + bias, k)[0], bias, dl)
    torch.cuda.synchronize()
    gr = torch.cuda.CUDAGraph()
    with torch.cuda.graph(gr):
        (d,) = torch.autograd.grad(autograd.moe_route(base + bias, k)[0], bias, dl)
    gr.replay()
    torch.cuda.synchronize()
    assert torch.equal(d, torch.autograd.grad(autograd.moe_route(base + bias, k)[0], bias, dl)[0])
    assert mxq.device_status() == 0


@pytest.mark.gpu
@pytest.mark.parametrize("E,k", [(4, 2), (20, 3), (60, 8), (300, 4)])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_a_token_beside_any_others(E, k, dtype):
    """Weights, choices and gradients of a token are the same bits whatever
    tokens stand beside it: far from zero, infinite, NaN, padded, or none."""
    T = 150
    l = logits_of(T, E, dtype, E)
    odd = torch.zeros(T, dtype=torch.bool)
    odd[::7] = True
    valid = torch.ones(T, dtype=torch.bool)
    valid[::21] = False
    gw = torch.randn(T, k, generator=torch.Generator().manual_seed(2))
    far = l.clone()
    rows = far[odd]
    for i in range(rows.shape[0]):
        rows[i] = (rows[i] + 2e6, rows[i] - 1e30, rows[i] * math.inf, rows[i] * math.nan, rows[i] * 1e9, rows[i] - math.inf)[i % 6]
    far[odd] = rows

    def run(l, valid, gw, renorm):
        x = l.to(DEV).requires_grad_(True)
        w, ids, _, _ = autograd.moe_route(x, k, valid=valid.to(DEV), renormalize=renorm)
        return w.detach(), ids, torch.autograd.grad(w, x, gw.to(DEV))[0]

    for renorm in (False, True):
        want = run(l[~odd], valid[~odd], gw[~odd], renorm)
        for got in (run(l, valid, gw, renorm), run(far, valid, gw, renorm)):
            for a, b in zip(got, want):
                assert torch.equal(a[~odd], b)
    assert mxq.device_status() == 0


@pytest.mark.gpu
@pytest.mark.parametrize("renorm", [False, True])
def test_a_bad_token_through_the_layer(renorm):
    """A token with a NaN or +inf among its logits: NaN weights, loss and logit
    gradients, zeros out of the layer, no trace in the other tokens."""
    T, E, k, K = 50, 8, 2, 96
    l = torch.randn(T, E, device=DEV)
    x = torch.randn(T, K, device=DEV)
    bad = torch.zeros(T, dtype=torch.bool, device=DEV)
    bad[[0, 17, 49]] = True
    l[0, 3], l[17, 0], l[49, 7] = math.nan, math.inf, math.nan
    dout = torch.randn(T, K, device=DEV)

    def layer(l, x, d):
        l, x = l.clone().requires_grad_(True), x.clone().requires_grad_(True)
        w, ids, counts, loss = autograd.moe_route(l, k, renormalize=renorm)
        xs, pos, offs = autograd.moe_dispatch(x, ids, E)
        out = autograd.moe_combine(2 * xs, pos, w, offs)
        return w, ids, counts, loss, out, *torch.autograd.grad(out, (l, x), d)

    w, ids, counts, loss, out, dl, dx = layer(l, x, dout)
    assert bool((ids[bad] == -1).all()) and bool(w[bad].isnan().all()) and bool(loss.isnan())
    assert bool((out[bad] == 0).all()) and bool((dx[bad] == 0).all()) and bool(dl[bad].isnan().all())
    alone = layer(l[~bad], x[~bad], dout[~bad])
    assert torch.equal(counts, alone[2]) and torch.equal(ids[~bad], alone[1])
    for got, want in zip((w, out, dl, dx), (alone[0], *alone[4:])):
        assert torch.equal(got[~bad], want)
    # weights of dropped slots count for nothing
    xs, pos, offs = autograd.moe_dispatch(x, ids, E)
    ww = torch.where(pos < 0, torch.full_like(w, math.inf), w)
    assert torch.equal(mxq.moe_combine(2 * xs, pos, ww), out) and torch.equal(mxq.moe_combine(2 * xs, pos, w), out)
    assert mxq.device_status() == 0


@pytest.mark.gpu
@pytest.mark.parametrize("T,E,k", [(2000000, 8, 2), (40000003, 4, 1), (1500001, 64, 3), (6000000, 256, 8), (1000000, 1000, 2)])
@pytest.mark.parametrize("alike", [False, True])
def test_loss_of_many_tokens(T, E, k, alike):
    """Sums of p over the tokens: a lane adds its tokens in fp32 (n of them, all
    terms positive, so n 2^-24 of the sum at most, and 16 more for the lanes and
    warps of a CTA), the CTAs are added in fp64; p is good to 2^-18. n is the
    tokens over 2 CTAs per SM, 16 warps each, 32 / lanes tokens at a time.
    `alike`: the same token throughout, whose roundings all go one way."""
    lanes = 1
    while lanes < 32 and lanes * 8 < E:
        lanes *= 2
    g = torch.Generator(device=DEV).manual_seed(E)
    if alike:
        l = (torch.randn(1, E, generator=g, device=DEV) * 2).bfloat16().expand(T, E).contiguous()
    else:
        l = torch.randn(T, E, generator=g, device=DEV, dtype=torch.bfloat16)
    w, ids, counts, loss = mxq.moe_route(l, k)
    assert int(counts.sum()) == T * k
    total = torch.zeros(E, dtype=torch.float64, device=DEV)
    seen = torch.zeros(E, dtype=torch.int64, device=DEV)
    for a, i in zip(l.split(1 << 18), ids.split(1 << 18)):
        total += torch.softmax(a.double(), 1).sum(0)
        seen += torch.bincount(i.reshape(-1), minlength=E)
    assert torch.equal(counts.long(), seen)
    want = E * float((seen.double() * total).sum()) / (k * float(T) ** 2)
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    n = math.ceil(T / (2 * sms * 16 * (32 // lanes)))
    assert abs(float(loss) - want) <= ((n + 17) * 2.0 ** -24 + 2.0 ** -18) * want
    assert mxq.device_status() == 0


@pytest.mark.gpu
@pytest.mark.parametrize("T,E,k", [(4097, 8, 4), (20000, 1000, 3), (40000, 37, 8)])
def test_orders_back_to_back(T, E, k):
    """The ranking kernel starts while the counting one still runs, and its
    workspace is the one of the call before: counts of another call's ids must
    not show."""
    L = mxq.lib()
    n = T * k
    batches = [torch.randint(-1, e, (T, k), device=DEV, dtype=torch.int32) for e in (E, 1, E // 2 + 1, 3, E, 2)]
    want = [mxq.moe_dispatch_plan(b, E) for b in batches]
    for b, (pos, offs) in zip(batches, want):
        key = torch.where(b < 0, E, b).reshape(-1).long()
        assert torch.equal(offs.long(), torch.cumsum(torch.bincount(key, minlength=E + 1)[:E], 0))
        order = torch.sort(key, stable=True).indices[:int(offs[-1])]
        assert torch.equal(pos.reshape(-1)[order].long(), torch.arange(order.numel(), device=DEV))
    nbytes = L.moe_dispatch_plan_workspace_bytes(n, E)
    assert nbytes > 0
    ws = torch.empty(nbytes, dtype=torch.uint8, device=DEV)
    reps = 20
    pos = torch.empty(reps * len(batches), T, k, dtype=torch.int32, device=DEV)
    offs = torch.empty(reps * len(batches), E, dtype=torch.int32, device=DEV)
    stream = torch.cuda.current_stream().cuda_stream
    for i in range(reps * len(batches)):
        assert L.moe_dispatch_plan(batches[i % len(batches)].data_ptr(), n, E, pos[i].data_ptr(), offs[i].data_ptr(),
                                   ws.data_ptr(), nbytes, stream) == mxq.OK
    for i in range(reps * len(batches)):
        assert torch.equal(pos[i], want[i % len(batches)][0]) and torch.equal(offs[i], want[i % len(batches)][1])
    assert mxq.device_status() == 0


@pytest.mark.gpu
def test_the_largest_order():
    """2^31 - 1 entries, the most that int32 places and ends can hold: against
    running counts, a part of the entries at a time."""
    n, E = 2 ** 31 - 1, 5
    ids = torch.empty(n, 1, dtype=torch.int32, device=DEV)
    g = torch.Generator(device=DEV).manual_seed(1)
    for part in ids.split(1 << 27):
        part.copy_(torch.randint(-1, E, part.shape, generator=g, device=DEV, dtype=torch.int32))
    pos, offs = mxq.moe_dispatch_plan(ids, E)
    counts = torch.zeros(E, dtype=torch.int64, device=DEV)
    for part in ids.split(1 << 27):
        counts += torch.stack([(part == e).sum() for e in range(E)])
    ends = torch.cumsum(counts, 0)
    assert torch.equal(offs.long(), ends)
    first = (ends - counts).tolist()
    for part, got in zip(ids.split(1 << 26), pos.split(1 << 26)):
        assert bool((got[part < 0] == -1).all())
        for e in range(E):
            mine = got[part == e]
            assert torch.equal(mine.long(), torch.arange(first[e], first[e] + mine.numel(), device=DEV))
            first[e] += mine.numel()
    assert first == ends.tolist()
    assert mxq.device_status() == 0


@pytest.mark.gpu
def test_the_most_tokens():
    """Tokens up to the limit of 2^31 - 1 slots through every call, in rows of
    one or two elements."""
    T, E, k = 2 ** 30 - 11, 2, 2  # 2^31 - 22 slots, 2^31 - 16 rows
    l = torch.empty(T, E, dtype=torch.bfloat16, device=DEV)
    bits = torch.arange(T, device=DEV, dtype=torch.int32)
    l[:, 0] = (bits & 1).bfloat16()
    l[:, 1] = (bits & 2).bfloat16()
    w, ids, counts, loss = mxq.moe_route(l, k)
    assert counts.tolist() == [T, T]
    four = mxq.moe_route(l[:4], k)
    tail = slice(T - T % 4 - 4, T - T % 4)
    for got, want in ((w, four[0]), (ids, four[1])):
        assert torch.equal(got[tail], want) and torch.equal(got[:4], want)
    p = torch.softmax(l[:4].double(), 1).mean(0)
    assert abs(float(loss) - float(p.sum())) <= 2.0 ** -9
    del l, w
    pos, offs = mxq.moe_dispatch_plan(ids, E)
    assert offs.tolist() == [T, 2 * T]
    assert torch.equal(pos[-4:].sort(1).values.long(), torch.arange(T - 4, T, device=DEV)[:, None] + torch.tensor([0, T], device=DEV))
    del ids
    x = (bits % 256)[:, None].bfloat16()
    xs = mxq.moe_dispatch(x, pos, offs)
    assert xs.shape[0] == 2 * T + 6 and bool((xs[2 * T:] == 0).all())
    for half in (xs[:T], xs[T:2 * T]):
        assert torch.equal(half, x)
    with pytest.raises(mxq.MXQError):  # 2^31 - 10 slots would make 2^31 rows
        mxq.moe_dispatch(torch.zeros(2 ** 30 - 5, 1, device=DEV), torch.zeros(2 ** 30 - 5, 2, dtype=torch.int32, device=DEV), offs)
    out = mxq.moe_combine(xs, pos)
    assert torch.equal(out, 2 * x)
    ww = torch.full((T, k), 0.5, device=DEV)
    dy, dw = mxq.moe_combine_backward(x, xs, pos, ww, offs)
    assert torch.equal(dy, 0.5 * xs) and torch.equal(dw[:, 0], x[:, 0].float().square()) and torch.equal(dw[:, 1], dw[:, 0])
    assert mxq.device_status() == 0
