"""The layer norm (ssd_layer_norm_fwd, ssd_layer_norm_bwd) against its 64-bit
form, element by element, within the bounds of tests/_ops_ref.py; its refusals;
and a block of norm, gated linear recurrence and gated output norm run
together, forward and backward."""
import ctypes

import pytest

torch = pytest.importorskip("torch")

import mamba_ssd_layer_fwd_b200 as ssd  # noqa: E402
from _ops_ref import Glr, Norm, assert_within, half_step  # noqa: E402

IO = {"bf16": torch.bfloat16, "f32": torch.float32}
gpu = pytest.mark.gpu


def make(shape, io, groups=1, kind="plain", bias=True, strided=False, seed=0, mean=0.3, device="cuda"):
    gen = torch.Generator().manual_seed(seed)
    D = shape[-1]
    rand = lambda *s: torch.randn(s, generator=gen)

    def rows():
        if not strided:
            return rand(*shape).to(device, IO[io])
        return rand(*shape[:-1], D + 11).to(device, IO[io])[..., 3:3 + D]

    return dict(x=rows() + torch.tensor(mean, dtype=IO[io]).to(device) if not strided else rows(),
                weight=(1 + 0.5 * rand(D)).to(device), bias=(0.3 * rand(D)).to(device) if bias else None,
                z=(rows() if kind == "gate" else None),
                res=rand(*shape).to(device, IO[io]) if kind == "residual" else None,
                dy=rand(*shape).to(device, IO[io]), dres=rand(*shape).to(device) if kind == "residual" else None,
                G=groups)


def fwd(p, eps=1e-5):
    out = ssd.ssd_layer_norm_fwd(p["x"], p["weight"], p["bias"], residual=p["res"], z=p["z"], ngroups=p["G"], eps=eps,
                                 return_stats=True)
    return out if p["res"] is not None else (out[0], None) + tuple(out[1:])


def check(p, eps=1e-5, device="cpu"):
    to = lambda v: None if v is None else v.to(device)
    ref = Norm(to(p["x"]), to(p["weight"]), to(p["bias"]), to(p["res"]), to(p["z"]), p["G"], eps)
    y, total, mean, rstd = fwd(p, eps)
    assert_within("y", y, ref.y, ref.ey)
    assert_within("mean", mean, ref.mean[..., 0], ref.emean[..., 0])
    assert_within("rstd", rstd, ref.rstd[..., 0], ref.erstd[..., 0])
    x = p["x"]
    if total is not None:
        assert torch.equal(total, (x.float() + p["res"].float()).to(x.dtype))
        x = total
    for gdt in {torch.float32, x.dtype}:
        dres = None if p["dres"] is None else p["dres"].to(gdt)
        got = ssd.ssd_layer_norm_bwd(x, p["weight"], p["dy"], mean, rstd, z=p["z"], dresidual=dres, ngroups=p["G"],
                                     grad_dtype=gdt)
        for k, (v, e) in ref.grad(to(p["dy"]), to(mean), to(rstd), to(dres)).items():
            assert got[k].dtype == (gdt if k in ("dx", "dz") else torch.float32)
            assert_within(f"{k} {gdt}", got[k], v, e)


# ------------------------------------------------------------------ CPU

def test_reference_against_torch_autograd():
    for kind, groups in (("plain", 1), ("plain", 3), ("gate", 4), ("residual", 1)):
        p = make((5, 12), "f32", groups, kind, device="cpu")
        d = {k: v.double() if torch.is_tensor(v) else v for k, v in p.items()}
        leaf = {k: d[k].clone().requires_grad_() for k in ("x", "weight", "bias", "z") if d[k] is not None}
        u = leaf["x"] if kind != "residual" else leaf["x"] + d["res"]
        v = u * torch.nn.functional.silu(leaf["z"]) if kind == "gate" else u
        y = torch.nn.functional.group_norm(v, groups, leaf["weight"], leaf["bias"], 1e-5)
        loss = (y * d["dy"]).sum() + (0 if kind != "residual" else (u * d["dres"]).sum())
        loss.backward()
        ref = Norm(d["x"], d["weight"], d["bias"], d["res"], d["z"], groups)
        if kind != "residual":                        # there the reference rounds the sum to float32
            assert torch.allclose(ref.y, y.detach(), rtol=0, atol=1e-12)
        ref.u = ref._split(v.detach())
        g = ref.grad(d["dy"], ref._split(v.detach()).mean(-1), (ref._split(v.detach()).var(-1, unbiased=False) + 1e-5).rsqrt(),
                     d["dres"])
        for k, n in (("dx", "x"), ("dweight", "weight"), ("dbias", "bias"), ("dz", "z")):
            if n in leaf:
                assert torch.allclose(g[k][0], leaf[n].grad, rtol=0, atol=1e-11), (kind, k)


def _meta(*shape, dtype=torch.bfloat16):
    return torch.empty(shape, dtype=dtype, device="meta")


def test_binding_checks():
    f32 = torch.float32
    ok = dict(x=_meta(3, 5, 24), weight=_meta(24, dtype=f32), bias=_meta(24, dtype=f32))
    assert ssd._validate_layer_norm(**ok) == (15, 24, 24, 24)
    assert ssd._validate_layer_norm(**ok, z=_meta(3, 5, 60)[..., 7:31], ngroups=4) == (15, 24, 24, 60)
    assert ssd._validate_layer_norm(**ok, residual=_meta(3, 5, 24))[0] == 15
    for name, bad in [("x", _meta(3, 5, 48)[..., ::2]), ("weight", None), ("weight", _meta(24)), ("bias", _meta(23, dtype=f32)),
                      ("z", _meta(3, 5, 25)), ("z", _meta(3, 5, 24, dtype=f32)), ("residual", _meta(3, 24)),
                      ("residual", _meta(3, 5, 60)[..., 7:31]), ("y", _meta(3, 5, 24, dtype=f32)), ("ngroups", 5),
                      ("ngroups", 0), ("x", _meta(3, 5, 0)), ("z", _meta(24).expand(3, 5, 24)),
                      ("x", torch.empty(3, 5, 24, dtype=torch.bfloat16))]:
        with pytest.raises(ValueError):
            ssd._validate_layer_norm(**dict(ok, **{name: bad}))
    with pytest.raises(ValueError, match="exclude"):
        ssd._validate_layer_norm(**ok, residual=_meta(3, 5, 24), z=_meta(3, 5, 24))
    with pytest.raises(TypeError):
        ssd._validate_layer_norm(_meta(3, 24, dtype=torch.float16), ok["weight"])
    b = dict(x=_meta(7, 24), weight=_meta(24, dtype=f32), dy=_meta(7, 24), mean=_meta(7, 4, dtype=f32),
             rstd=_meta(7, 4, dtype=f32), ngroups=4)
    assert ssd._validate_layer_norm_bwd(**b)[:2] == (7, 24)
    assert ssd._validate_layer_norm_bwd(**b, dresidual=_meta(7, 24, dtype=f32))[4] == f32
    assert ssd._validate_layer_norm_bwd(**b, dresidual=_meta(7, 24), grad_dtype=torch.bfloat16)[4] == torch.bfloat16
    for name, bad in [("dy", None), ("dy", _meta(7, 24, dtype=f32)), ("mean", _meta(7, 1, dtype=f32)), ("rstd", None),
                      ("rstd", _meta(7, 4)), ("dresidual", _meta(7, 24)), ("grad_dtype", torch.float64)]:
        with pytest.raises(ValueError):
            ssd._validate_layer_norm_bwd(**dict(b, **{name: bad}))
    with pytest.raises(ValueError, match="exclude"):
        ssd._validate_layer_norm_bwd(**b, z=_meta(7, 24), dresidual=_meta(7, 24, dtype=f32))
    with pytest.raises(ValueError, match="CUDA"):
        ssd.ssd_layer_norm_fwd(b["x"], b["weight"])


def test_abi_refuses_before_any_launch():
    lib = ssd.library()

    def params(rows=7, dim=24, groups=4, eps=1e-5, io=1, grad=1, xs=24, zs=24):
        return ssd.SsdLayerNormParams(rows, dim, groups, eps, io, grad, xs, zs)

    def f(p, x=16, res=None, z=None, w=16, b=16, y=16, total=None, mean=16):
        return lib.ssd_layer_norm_fwd(ctypes.byref(p), x, res, z, w, b, y, total, mean, 16, None)

    def g(p, x=16, z=None, w=16, mean=16, dy=16, dres=None, dx=16, dz=None, dw=16, db=16, ws=256, n=1 << 40):
        return lib.ssd_layer_norm_bwd(ctypes.byref(p), x, z, w, mean, 16, dy, dres, dx, dz, dw, db, ws, n, None)

    for bad in (dict(rows=-1), dict(dim=0), dict(groups=0), dict(groups=5), dict(eps=-1.0), dict(eps=float("nan")),
                dict(io=2), dict(io=0), dict(xs=23)):
        assert f(params(**bad)) == -1 and g(params(**bad)) == -1, bad
        assert lib.ssd_layer_norm_bwd_workspace_size(ctypes.byref(params(**bad))) == 0
    for bad in (dict(rows=1 << 31), dict(dim=16385, groups=1, xs=16385), dict(xs=1 << 31)):
        assert f(params(**bad)) == -2 and g(params(**bad)) == -2, bad
    assert lib.ssd_layer_norm_fwd(None, *[16] * 9, None) == -1
    for bad in (dict(x=None), dict(w=None), dict(y=None), dict(x=1), dict(w=2), dict(mean=2), dict(res=16),
                dict(total=16), dict(res=16, total=16, z=16)):
        assert f(params(), **bad) == -1, bad
    assert f(params(zs=23), z=16) == -1
    for bad in (dict(x=None), dict(w=None), dict(mean=None), dict(dy=None), dict(dx=None), dict(dw=None), dict(z=16),
                dict(dz=16), dict(z=16, dz=16, dres=16), dict(ws=None), dict(ws=16), dict(n=4), dict(dy=1), dict(db=2)):
        assert g(params(), **bad) == -1, bad
    assert f(params(rows=0), x=None, y=None) == 0


# ------------------------------------------------------------------ GPU

@gpu
@pytest.mark.parametrize("io", ["bf16", "f32"])
@pytest.mark.parametrize("kind", ["plain", "residual", "gate"])
@pytest.mark.parametrize("shape,groups", [((1, 1), 1), ((3, 7), 1), ((5, 64), 1), ((2, 3, 264), 1), ((300, 72), 1),
                                          ((7, 1027), 1), ((9, 1536), 24), ((4, 183), 3), ((33, 2560), 1),
                                          ((20, 320), 5), ((6, 4104), 1), ((5, 2048), 2), ((700, 96), 1),
                                          ((3, 8200), 1), ((2, 5001), 1), ((11, 130), 130)])
def test_values(io, kind, shape, groups):
    check(make(shape, io, groups, kind, bias=shape[0] != 9, strided=shape[0] in (3, 4, 20), seed=sum(shape)))


@gpu
@pytest.mark.parametrize("io", ["bf16", "f32"])
@pytest.mark.parametrize("D", [16384, 16383, 12000])
def test_longest_groups(io, D):
    check(make((3, D), io, 1, "plain", seed=D))
    check(make((2, D), io, 1, "gate", seed=D))


@gpu
@pytest.mark.parametrize("io", ["bf16", "f32"])
def test_many_rows(io):
    check(make((5000, 520), io, 1, "residual", seed=1), device="cuda")
    check(make((3001, 640), io, 10, "gate", seed=2), device="cuda")


@gpu
@pytest.mark.parametrize("io", ["bf16", "f32"])
@pytest.mark.parametrize("kind", ["plain", "residual", "gate"])
@pytest.mark.parametrize("shape,groups", [((3001, 1544), 1), ((2403, 2560), 1), ((1501, 5120), 1), ((700, 8192), 2),
                                          ((1600, 6152), 1)])
def test_many_long_rows(io, kind, shape, groups):
    """Rows enough that a CTA walks several of them."""
    check(make(shape, io, groups, kind, seed=shape[0]), device="cuda")


@gpu
@pytest.mark.parametrize("io", ["bf16", "f32"])
@pytest.mark.parametrize("rows,D,groups", [(2500, 1280, 1), (900, 640, 10), (2000, 512, 1)])
def test_columns_of_a_wider_tensor(io, rows, D, groups):
    """x and z as aligned column ranges of one tensor, forward and backward."""
    p = make((rows, D), io, groups, "gate", seed=D)
    wide = torch.cat([p["x"], p["dy"], p["z"]], -1)
    p["x"], p["z"] = wide[:, :D], wide[:, 2 * D:]
    check(p, device="cuda")


@gpu
def test_offsets_beyond_32_bits():
    rows, D, stride = 20000, 64, 110000
    assert (rows - 1) * stride > 2 ** 31
    p = make((rows, D), "bf16", 2, "gate", seed=31)
    big = torch.empty(rows * stride, dtype=torch.bfloat16, device="cuda").view(rows, stride)
    big[:, 16:16 + D], big[:, 512:512 + D] = p["x"], p["z"]
    p["x"], p["z"] = big[:, 16:16 + D], big[:, 512:512 + D]
    check(p, device="cuda")


@gpu
def test_a_row_far_from_zero_and_a_row_of_one_value():
    p = make((6, 1000), "f32", seed=3)
    p["x"][0] += 1000.0                       # mean far above the spread
    p["x"][1] = 3.0                           # no spread at all: rstd = 1 / sqrt(eps), y = bias
    p["x"][2, 0] = 4000.0                     # one outlier
    p["x"][3] = 0.0
    check(p)
    y = fwd(p)[0]
    assert torch.equal(y[1], p["bias"]) and torch.equal(y[3], p["bias"])


@gpu
def test_gates_at_their_ends():
    p = make((40, 256), "f32", 4, "gate", seed=4)
    p["z"][0], p["z"][1], p["z"][2, :7], p["z"][3, ::2] = 100.0, -100.0, -1000.0, 88.0
    to = lambda v: v.cpu()
    ref = Norm(to(p["x"]), to(p["weight"]), to(p["bias"]), None, to(p["z"]), 4)
    y, _, mean, rstd = fwd(p)
    for v in (y, mean, rstd, *ssd.ssd_layer_norm_bwd(p["x"], p["weight"], p["dy"], mean, rstd, z=p["z"], ngroups=4).values()):
        assert bool(torch.isfinite(v).all())
    assert_within("y", y[4:], ref.y[4:], ref.ey[4:])
    assert_within("y", y[:1], ref.y[:1], ref.ey[:1])


@gpu
def test_a_row_that_is_not_finite_leaves_the_others_alone():
    p = make((70, 640), "bf16", 10, "gate", seed=5)
    y0, _, m0, r0 = fwd(p)
    g0 = ssd.ssd_layer_norm_bwd(p["x"], p["weight"], p["dy"], m0, r0, z=p["z"], ngroups=10)
    p["x"][33], p["dy"][33] = float("nan"), float("inf")
    y, _, m, r = fwd(p)
    g = ssd.ssd_layer_norm_bwd(p["x"], p["weight"], p["dy"], m, r, z=p["z"], ngroups=10)
    rest = [k for k in range(70) if k != 33]
    for a, b in ((y, y0), (m, m0), (r, r0), (g["dx"], g0["dx"]), (g["dz"], g0["dz"])):
        assert torch.equal(a[rest], b[rest])


@gpu
def test_no_rows():
    x = torch.empty((0, 24), dtype=torch.bfloat16, device="cuda")
    w = torch.ones(24, device="cuda")
    y, mean, rstd = ssd.ssd_layer_norm_fwd(x, w, return_stats=True)
    assert y.shape == (0, 24) and mean.shape == (0, 1)
    g = ssd.ssd_layer_norm_bwd(x, w, x, mean, rstd)
    assert g["dx"].shape == (0, 24) and not g["dweight"].any() and not g["dbias"].any()


@gpu
@pytest.mark.parametrize("kind,groups", [("residual", 1), ("gate", 20)])
def test_the_same_call_gives_the_same_bits_on_any_stream_and_in_a_graph(kind, groups):
    p = make((2000, 1280), "bf16", groups, kind, seed=6)
    ws = torch.full((1 << 24,), 0xFF, dtype=torch.uint8, device="cuda")

    def both(**kw):
        y, total, mean, rstd = fwd(p)
        g = ssd.ssd_layer_norm_bwd(p["x"], p["weight"], p["dy"], mean, rstd, z=p["z"], dresidual=p["dres"], ngroups=groups, **kw)
        return [v for v in (y, total, mean, rstd, *g.values()) if v is not None]

    want = both()
    torch.cuda.synchronize()
    outs = [both(workspace=ws)]
    for s in [torch.cuda.Stream() for _ in range(2)]:
        with torch.cuda.stream(s):
            outs += [both() for _ in range(2)]
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        outs.append(both())
    for _ in range(2):
        graph.replay()
    torch.cuda.synchronize()
    for o in outs:
        assert all(torch.equal(a, b) for a, b in zip(o, want))


@gpu
@pytest.mark.parametrize("io,tol", [("f32", 1e-4), ("bf16", 2e-2)])
def test_gate_form_is_the_norm_that_ssd_fwd_applies(io, tol):
    """ssd_fwd followed by the norm with a gate and one group a head equals ssd_fwd given z: each is within
    the forward's tolerance (1e-4 float32, 2e-2 bf16 of the largest value) of the same result."""
    from _helpers import small_inputs, to_device
    t = to_device(small_inputs(batch=2, seqlen=300, H=4, P=64, N=64, io=io, seed=11))
    gen = torch.Generator(device="cuda").manual_seed(1)
    z = torch.randn(t["x"].shape, generator=gen, device="cuda").to(t["x"].dtype)
    w = torch.rand(256, generator=gen, device="cuda") + 0.5
    b = torch.randn(256, generator=gen, device="cuda") * 0.1
    args = (t["x"], t["dt"], t["A_log"], t["B"], t["C"], t["D"])
    want = ssd.ssd_fwd(*args, initial_states=t["initial_states"], z=z, norm_weight=w, norm_bias=b)
    y = ssd.ssd_fwd(*args, initial_states=t["initial_states"])
    got = ssd.ssd_layer_norm_fwd(y.view(2, 300, 256), w, b, z=z.view(2, 300, 256), ngroups=4)
    d = (got.double() - want.view(2, 300, 256).double()).abs().max() / want.double().abs().max()
    assert float(d) <= 2 * tol


@gpu
@pytest.mark.parametrize("io", ["bf16", "f32"])
def test_block_forward_and_backward(io):
    """norm(x + residual) -> one projection to (x, r, i, z) -> gated linear recurrence -> gated output norm, and
    back, as a training step calls them: gradients against autograd in 64 bits."""
    dt = IO[io]
    b, T, d, D, H = 2, 150, 48, 96, 6
    gen = torch.Generator().manual_seed(12)
    rand = lambda *s, std=1.0: (torch.randn(s, generator=gen) * std).cuda()
    x, res, dy = rand(b, T, d).to(dt), rand(b, T, d).to(dt), rand(b, T, D).to(dt)
    W = rand(d, 4 * D, std=d ** -0.5).to(dt)
    w1, b1, w2, b2 = 1 + rand(d, std=0.1), rand(d, std=0.1), 1 + rand(D, std=0.1), rand(D, std=0.1)
    A = rand(D, std=0.5) - 2.0

    n1, total, m1, r1 = ssd.ssd_layer_norm_fwd(x, w1, b1, residual=res, return_stats=True)
    proj = n1 @ W
    xs, rs, is_, zs = proj.split(D, -1)
    h, kept = ssd.ssd_glr_fwd(xs, rs, is_, A, return_chunk_states=True)
    out, m2, r2 = ssd.ssd_layer_norm_fwd(h, w2, b2, z=zs, ngroups=H, return_stats=True)
    g2 = ssd.ssd_layer_norm_bwd(h, w2, dy, m2, r2, z=zs, ngroups=H, grad_dtype=dt)
    gr = ssd.ssd_glr_bwd(xs, rs, is_, A, g2["dx"], chunk_states=kept, grad_dtype=dt)
    dproj = torch.cat([gr["dx"], gr["dr"], gr["di"], g2["dz"]], -1)
    g1 = ssd.ssd_layer_norm_bwd(total, w1, dproj @ W.t(), m1, r1, dresidual=torch.zeros_like(x).to(dt), grad_dtype=dt)

    leaf = {k: v.double().requires_grad_() for k, v in dict(x=x, w1=w1, b1=b1, w2=w2, b2=b2, A=A, W=W).items()}
    u = leaf["x"] + res.double()
    q = torch.nn.functional.layer_norm(u, (d,), leaf["w1"], leaf["b1"], 1e-5) @ leaf["W"]
    X, R, I, Z = q.split(D, -1)
    rate = leaf["A"].exp() * torch.sigmoid(R)
    s, hs = torch.zeros(b, D, dtype=torch.float64, device="cuda"), []
    for t in range(T):
        s = torch.exp(-rate[:, t]) * s + torch.sqrt(-torch.expm1(-2 * rate[:, t])) * torch.sigmoid(I[:, t]) * X[:, t]
        hs.append(s)
    v = (torch.stack(hs, 1) * torch.nn.functional.silu(Z)).reshape(b * T, D)
    o = torch.nn.functional.group_norm(v, H, leaf["w2"], leaf["b2"], 1e-5).view(b, T, D)
    (o * dy.double()).sum().backward()
    # Seven roundings to dt lie between the input and the furthest gradient (sum, norm, projection, state, two
    # gradients, their product), each half a step of the values around it, and the norms divide by a spread of order
    # one; in the 2-norm they add to less than 7 * 4 half steps (float32: plus sums over 48..300 terms, 2^6 half steps).
    lim = (28 + (64 if io == "f32" else 0)) * half_step(dt)
    near = lambda a, c: float((a.double() - c).norm() / c.norm())
    pairs = dict(out=(out, o.detach()), dx=(g1["dx"], leaf["x"].grad), dw1=(g1["dweight"], leaf["w1"].grad),
                 db1=(g1["dbias"], leaf["b1"].grad), dw2=(g2["dweight"], leaf["w2"].grad),
                 db2=(g2["dbias"], leaf["b2"].grad), dA=(gr["dA_log"], leaf["A"].grad),
                 dW=((n1.reshape(-1, d).t() @ dproj.reshape(-1, 4 * D)), leaf["W"].grad))
    errs = {k: near(a, c) for k, (a, c) in pairs.items()}
    assert all(e <= lim for e in errs.values()), (lim, errs)
