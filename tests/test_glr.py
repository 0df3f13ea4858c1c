"""The gated linear recurrence (ssd_glr_fwd, ssd_glr_bwd, ssd_glr_step)
against its 64-bit form, element by element, within the bounds of
tests/_ops_ref.py; its refusals; and its behaviour on streams, in graphs and
with reused workspaces."""
import ctypes

import pytest

torch = pytest.importorskip("torch")

import mamba_ssd_layer_fwd_b200 as ssd  # noqa: E402
from _ops_ref import Glr, assert_within  # noqa: E402

IO = {"bf16": torch.bfloat16, "f32": torch.float32}
gpu = pytest.mark.gpu


def make(b, T, D, io, cu=None, strided=False, init=True, seed=0, lo=-4.8, hi=0.5, std=1.0, device="cuda"):
    gen = torch.Generator().manual_seed(seed)
    n = b if cu is None else len(cu) - 1
    rand = lambda *s: torch.randn(s, generator=gen)
    if strided:
        x, r, i = (rand(b, T, 3 * D + 5) * std).to(device, IO[io])[..., 2:2 + 3 * D].split(D, -1)
    else:
        x, r, i = ((rand(b, T, D) * std).to(device, IO[io]) for _ in range(3))
    return dict(x=x, r=r, i=i, A_log=(torch.rand(D, generator=gen) * (hi - lo) + lo).to(device),
                init=rand(n, D).to(device) if init else None, dfinal=rand(n, D).to(device) if init else None,
                dy=rand(b, T, D).to(device, IO[io]), cu=cu,
                cu_t=None if cu is None else torch.tensor(cu, dtype=torch.int32, device=device))


def ref_of(p, device="cpu"):
    to = lambda v: None if v is None else v.to(device)
    return Glr(to(p["x"]), to(p["r"]), to(p["i"]), to(p["A_log"]), to(p["init"]), p["cu"])


def fwd(p, **kw):
    return ssd.ssd_glr_fwd(p["x"], p["r"], p["i"], p["A_log"], initial_states=p["init"], cu_seqlens=p["cu_t"],
                           return_final_states=True, return_chunk_states=True, check_status=True, **kw)


def bwd(p, **kw):
    return ssd.ssd_glr_bwd(p["x"], p["r"], p["i"], p["A_log"], p["dy"], initial_states=p["init"],
                           cu_seqlens=p["cu_t"], dfinal_states=p["dfinal"], check_status=True, **kw)


def check(p, device="cpu"):
    ref = ref_of(p, device)
    y, final, chunks = fwd(p)
    assert_within("y", y, ref.h, ref.eh)
    assert_within("final", final, ref.final, ref.efinal)
    assert_within("chunk states", chunks, ref.chunks, ref.echunks)
    want = ref.grad(p["dy"].to(device), p["dfinal"])
    dtypes = (torch.float32, p["x"].dtype) if p["x"].dtype != torch.float32 else (torch.float32,)
    for gdt in dtypes:
        for kept in (chunks, None):
            got = bwd(p, chunk_states=kept, grad_dtype=gdt)
            for k, (v, e) in want.items():
                assert got[k].dtype == (gdt if k in ("dx", "dr", "di") else torch.float32)
                assert_within(f"{k} {gdt} kept={kept is not None}", got[k], v, e)


# ------------------------------------------------------------------ CPU: the reference, refusals

def test_reference_gradient_against_differences():
    p = make(1, 7, 3, "f32", cu=[0, 3, 3, 7], device="cpu")
    p = {k: v.double() if torch.is_tensor(v) and v.is_floating_point() else v for k, v in p.items()}
    loss = lambda q: float((lambda f: (f.h * q["dy"]).sum() + (f.final * q["dfinal"]).sum())(ref_of(q)))
    got = ref_of(p).grad(p["dy"], p["dfinal"])
    for name, key in (("x", "dx"), ("r", "dr"), ("i", "di"), ("A_log", "dA_log"), ("init", "dinitial_states")):
        flat = p[name].reshape(-1)
        for k in range(flat.numel()):
            vals = []
            for step in (1e-5, -1e-5):
                v = flat.clone()
                v[k] += step
                vals.append(loss(dict(p, **{name: v.view_as(p[name])})))
            # central difference: third derivatives of order 1 times 1e-10, rounding 1e-16 / 1e-5
            assert abs((vals[0] - vals[1]) / 2e-5 - float(got[key][0].reshape(-1)[k])) < 1e-8, (name, k)


def test_reference_against_a_hand_worked_value():
    # r = 0, exp(A_log) = 2 ln 2: q = ln 2, a = 1/2, m = sqrt(3)/2; i = 0: h = h0/2 + sqrt(3)/4 x
    z = torch.zeros(1, 2, 1)
    A = torch.log(2 * torch.log(torch.tensor([2.0], dtype=torch.float64)))
    f = Glr(torch.tensor([[[4.0], [0.0]]]), z, z, A, torch.tensor([[8.0]]))
    assert abs(float(f.h[0, 0]) - (4 + 3 ** 0.5)) < 1e-14
    assert abs(float(f.h[0, 1]) - (4 + 3 ** 0.5) / 2) < 1e-14


def _meta(*shape, dtype=torch.bfloat16):
    return torch.empty(shape, dtype=dtype, device="meta")


def test_binding_checks():
    f32, i32 = torch.float32, torch.int32
    ok = dict(x=_meta(2, 70, 24), r=_meta(2, 70, 24), i=_meta(2, 70, 24), A_log=_meta(24, dtype=f32),
              initial_states=_meta(2, 24, dtype=f32), y=_meta(2, 70, 24), final_states=_meta(2, 24, dtype=f32),
              chunk_states=_meta(2, 2, 24, dtype=f32), dy=_meta(2, 70, 24), dfinal_states=_meta(2, 24, dtype=f32))
    assert ssd._validate_glr(**ok) == (2, (24, 24, 24))
    x, r, i = _meta(2, 70, 72).split(24, -1)
    assert ssd._validate_glr(**dict(ok, x=x, r=r, i=i)) == (2, (72, 72, 72))
    assert ssd._validate_glr(_meta(2, 1, 72)[..., :24], *[_meta(2, 1, 24)] * 2, ok["A_log"])[1] == (72, 24, 24)
    for name, bad in [("r", _meta(2, 70, 25)), ("i", None), ("i", _meta(2, 70, 24, dtype=f32)),
                      ("x", _meta(2, 70, 48)[..., ::2]), ("r", _meta(2, 70, 1).expand(2, 70, 24)),
                      ("r", _meta(1, 70, 24).expand(2, 70, 24)), ("i", _meta(70, 2, 24).transpose(0, 1)),
                      ("x", _meta(2, 75, 24)[:, :70]), ("r", torch.empty(2, 70, 24, dtype=torch.bfloat16)),
                      ("A_log", None), ("A_log", _meta(24)), ("A_log", _meta(2, 24, dtype=f32)),
                      ("initial_states", _meta(1, 24, dtype=f32)), ("y", _meta(2, 70, 48)[..., :24]),
                      ("final_states", _meta(2, 24)), ("chunk_states", _meta(2, 1, 24, dtype=f32)),
                      ("dy", _meta(2, 70, 24, dtype=f32)), ("dfinal_states", _meta(2, 25, dtype=f32)),
                      ("cu_seqlens", _meta(3, dtype=i32)), ("x", _meta(70, 24))]:
        with pytest.raises(ValueError):
            ssd._validate_glr(**dict(ok, **{name: bad}))
    with pytest.raises(TypeError):
        ssd._validate_glr(**dict(ok, x=_meta(2, 70, 24, dtype=torch.float16)))
    one = dict(x=_meta(1, 9, 4), r=_meta(1, 9, 4), i=_meta(1, 9, 4), A_log=_meta(4, dtype=f32))
    assert ssd._validate_glr(**one, cu_seqlens=_meta(6, dtype=i32), initial_states=_meta(5, 4, dtype=f32))[0] == 5
    for cu in (_meta(1, dtype=i32), _meta(6, dtype=torch.int64), _meta(2, 3, dtype=i32)):
        with pytest.raises(ValueError):
            ssd._validate_glr(**one, cu_seqlens=cu)
    step = dict(x=_meta(5, 8), r=_meta(5, 8), i=_meta(5, 8), A_log=_meta(8, dtype=f32), state=_meta(5, 8, dtype=f32))
    assert ssd._validate_glr_step(**step) == (8, 8, 8)
    assert ssd._validate_glr_step(**dict(step, r=_meta(5, 24)[:, 8:16])) == (8, 24, 8)
    for name, bad in [("state", None), ("state", _meta(5, 8)), ("state", _meta(4, 8, dtype=f32)), ("y", _meta(5, 9)),
                      ("r", _meta(8).expand(5, 8)), ("A_log", _meta(9, dtype=f32)), ("x", _meta(5, 8, 1))]:
        with pytest.raises(ValueError):
            ssd._validate_glr_step(**dict(step, **{name: bad}))
    with pytest.raises(ValueError, match="grad_dtype"):
        ssd._grad_dtype(torch.float32, torch.bfloat16)
    with pytest.raises(ValueError, match="CUDA"):
        ssd.ssd_glr_fwd(one["x"], one["r"], one["i"], one["A_log"])


def test_abi_refuses_before_any_launch():
    lib = ssd.library()

    def params(batch=2, seqlen=70, channels=24, num_seqs=0, io=1, grad=0, xs=24, rs=24, i_s=24):
        return ssd.SsdGlrParams(batch, seqlen, channels, num_seqs, io, grad, xs, rs, i_s)

    def f(p, x=16, r=16, i=16, A=16, init=None, cu=None, y=16, ws=256, n=1 << 40):
        return lib.ssd_glr_fwd(ctypes.byref(p), x, r, i, A, init, cu, y, None, None, ws, n, None)

    def g(p, x=16, A=16, cu=None, chunks=16, dy=16, dx=16, dA=16, dfin=None, ws=256, n=1 << 40):
        return lib.ssd_glr_bwd(ctypes.byref(p), x, 16, 16, A, None, cu, chunks, dy, dfin, dx, 16, 16, dA, None, ws, n, None)

    for bad in (dict(batch=0), dict(seqlen=-1), dict(channels=0), dict(num_seqs=-1), dict(num_seqs=2), dict(io=2),
                dict(grad=2), dict(io=0, grad=1), dict(xs=23), dict(rs=0), dict(i_s=-24)):
        assert f(params(**bad)) == -1 and g(params(**bad)) == -1, bad
        assert lib.ssd_glr_fwd_workspace_size(ctypes.byref(params(**bad))) == 0
        assert lib.ssd_glr_bwd_workspace_size(ctypes.byref(params(**bad)), 0) == 0
    for bad in (dict(batch=70000, seqlen=70000), dict(xs=1 << 31), dict(batch=1, num_seqs=(1 << 20) + 1)):
        assert f(params(**bad), cu=16 if "num_seqs" in bad else None) == -2, bad
    assert lib.ssd_glr_fwd(None, 16, 16, 16, 16, None, None, 16, None, None, 256, 1 << 20, None) == -1
    for bad in (dict(x=None), dict(r=None), dict(A=None), dict(y=None), dict(ws=None), dict(ws=128), dict(n=8),
                dict(x=17), dict(y=1), dict(A=2), dict(init=6), dict(cu=16)):
        assert f(params(), **bad) == -1, bad
    assert f(params(batch=1, num_seqs=3)) == -1                       # cu_seqlens missing
    for bad in (dict(dy=None), dict(dx=None), dict(dA=None), dict(dx=2), dict(dfin=2), dict(chunks=2), dict(n=256),
                dict(chunks=None, n=lib.ssd_glr_bwd_workspace_size(ctypes.byref(params()), 1))):
        assert g(params(), **bad) == -1, bad

    def s(batch=3, channels=8, io=1, xs=8, x=16, state=16, y=16, A=16):
        return lib.ssd_glr_step(ctypes.byref(ssd.SsdGlrStepParams(batch, channels, io, xs, 8, 8)), x, 16, 16, A, state,
                                y, None)

    for bad in (dict(batch=-1), dict(channels=0), dict(io=3), dict(xs=7), dict(x=None), dict(state=None),
                dict(state=2), dict(y=1), dict(A=None)):
        assert s(**bad) == -1, bad
    assert s(batch=0, x=None, state=None) == 0


# ------------------------------------------------------------------ GPU: values

@gpu
@pytest.mark.parametrize("io", ["bf16", "f32"])
@pytest.mark.parametrize("b,T,D", [(1, 1, 1), (3, 1, 7), (2, 2, 64), (3, 63, 5), (2, 64, 66), (2, 65, 33), (1, 129, 130),
                                   (2, 513, 40), (5, 200, 264), (1, 4500, 3), (2, 1300, 72)])
def test_rows(io, b, T, D):
    check(make(b, T, D, io, strided=T % 2 == 1, init=D != 66, seed=T + D))


@gpu
@pytest.mark.parametrize("io", ["bf16", "f32"])
@pytest.mark.parametrize("lens,D", [([1, 255, 0, 97, 33, 3], 72), ([0, 0, 5, 0], 9), ([0], 4), ([64, 64, 1, 0, 63, 130], 128),
                                    ([1] * 70, 33), ([2000], 16), ([0, 700, 0, 0, 1333, 0], 64), ([128, 128, 256], 70)])
def test_packed(io, lens, D):
    cu = [0]
    for n in lens:
        cu.append(cu[-1] + n)
    check(make(1, cu[-1], D, io, cu=cu, strided=D % 2 == 1, init=D != 70, seed=D))


@gpu
@pytest.mark.parametrize("io", ["bf16", "f32"])
@pytest.mark.parametrize("b,T,D,lens", [(2, 200, 72, None), (1, 65, 33, None), (1, 0, 130, [64, 1, 0, 70, 300]),
                                        (4, 130, 4096, None), (1, 700, 40, [7] * 100)])
def test_rates_of_at_most_one(io, b, T, D, lens):
    """Rates of at most 1 have an arithmetic of their own; 4 x 4096 channels fill the SMs, which has shorter groups."""
    cu = None
    if lens:
        cu = [0]
        for n in lens:
            cu.append(cu[-1] + n)
    check(make(b, cu[-1] if cu else T, D, io, cu=cu, hi=0.0, lo=-6.0, seed=D), "cpu" if D < 1000 else "cuda")


@gpu
@pytest.mark.parametrize("io", ["bf16", "f32"])
def test_thirds_of_one_projection_and_offsets_beyond_32_bits(io):
    """x, r and i as column ranges: of one tensor, and of one whose last rows lie 2^31 elements behind its first."""
    D = 72
    p = make(2, 133, D, io, seed=21)
    proj = torch.cat([p["x"], p["r"], p["i"]], -1)
    p["x"], p["r"], p["i"] = proj.split(D, -1)
    check(p)
    T, stride = 20000, 110000
    p = make(1, T, D, io, seed=22, hi=0.0)
    big = torch.empty(T * stride, dtype=IO[io], device="cuda").view(1, T, stride)
    assert (T - 1) * stride > 2 ** 31
    big[..., 8:8 + 3 * D] = torch.cat([p["x"], p["r"], p["i"]], -1)
    want = fwd(p)
    grads = bwd(p, chunk_states=want[2])
    p["x"], p["r"], p["i"] = big[..., 8:8 + 3 * D].split(D, -1)
    assert all(torch.equal(a, b) for a, b in zip(fwd(p), want))
    got = bwd(p, chunk_states=want[2])
    assert all(torch.equal(got[k], grads[k]) for k in grads)


@gpu
def test_a_given_stream_and_a_call_after_it():
    p = make(2, 500, 64, "bf16", seed=23)
    want = fwd(p)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    got = ssd.ssd_glr_fwd(p["x"], p["r"], p["i"], p["A_log"], initial_states=p["init"], return_final_states=True,
                          return_chunk_states=True, stream=s)
    s.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))


@gpu
def test_many_sequences():
    """More sequences than a grid's second dimension holds, most of them empty."""
    n = 70000
    cu = sorted([0, 200] + [int(v) for v in torch.randint(0, 201, (n - 1,), generator=torch.Generator().manual_seed(3))])
    p = make(1, 200, 8, "f32", cu=cu)
    ref = ref_of(p)
    y, final, _ = fwd(p)
    assert_within("y", y, ref.h, ref.eh)
    assert_within("final", final, ref.final, ref.efinal)
    got = bwd(p)
    for k, (v, e) in ref.grad(p["dy"].cpu(), p["dfinal"]).items():
        assert_within(k, got[k], v, e)


@gpu
@pytest.mark.parametrize("io", ["bf16", "f32"])
def test_long_memory_rows_split_over_the_time_axis(io):
    """Rates down to 1e-4: the state carries over thousands of tokens."""
    check(make(2, 9000, 34, io, seed=5, lo=-9.2, hi=-2.0), "cuda")


@gpu
@pytest.mark.parametrize("io", ["bf16", "f32"])
def test_rates_and_gates_at_their_ends(io):
    p = make(2, 150, 12, io, seed=6)
    p["A_log"][:4] = torch.tensor([float("-inf"), 30.0, -20.0, 3.0])       # a = 1; a = 0; slow; fast
    g = torch.Generator().manual_seed(1)
    for k in ("r", "i"):
        v = p[k].clone()
        at = torch.randint(0, v.numel(), (600,), generator=g).cuda()
        v.view(-1)[at] = torch.where(torch.rand(600, generator=g).cuda() < 0.5, 30.0, -30.0).to(v.dtype)
        p[k] = v
    check(p)


@gpu
def test_zero_tokens():
    for cu in (None, [0, 0, 0]):
        p = make(1 if cu else 2, 0, 10, "bf16", cu=cu)
        y, final, chunks = fwd(p)
        assert y.shape == p["x"].shape and chunks.shape[1] == 0
        assert torch.equal(final, p["init"])
        got = bwd(p)
        assert torch.equal(got["dinitial_states"], p["dfinal"]) and not got["dA_log"].any()
    p["cu_t"] = torch.tensor([0, 3, 0], dtype=torch.int32, device="cuda")
    for call in (fwd, bwd):
        with pytest.raises(ssd.SsdError) as e:
            call(p)
        assert e.value.code == -5
    x = torch.empty((0, 6), dtype=torch.bfloat16, device="cuda")
    assert ssd.ssd_glr_step(x, x, x, torch.zeros(6, device="cuda"), torch.empty((0, 6), device="cuda")).shape == (0, 6)


@gpu
@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
def test_a_sequence_that_is_not_finite_leaves_the_others_alone(bad):
    cu = [0, 90, 100, 400, 401, 600]
    p = make(1, 600, 20, "f32", cu=cu, seed=7)
    y0, f0, _ = fwd(p)
    g0 = bwd(p)
    for k in ("x", "dy"):
        p[k] = p[k].clone()
        p[k][:, 100:400] = bad
    p["init"], p["dfinal"] = p["init"].clone(), p["dfinal"].clone()
    p["init"][2], p["dfinal"][2] = bad, bad
    y, f, _ = fwd(p)
    g = bwd(p)
    rest = [t for t in range(600) if not 100 <= t < 400]
    assert torch.equal(y[:, rest], y0[:, rest]) and torch.equal(f[[0, 1, 3, 4]], f0[[0, 1, 3, 4]])
    for k in ("dx", "dr", "di"):
        assert torch.equal(g[k][:, rest], g0[k][:, rest]), k
    assert torch.equal(g["dinitial_states"][[0, 1, 3, 4]], g0["dinitial_states"][[0, 1, 3, 4]])
    assert not torch.isfinite(y[:, 100:400]).any()


@gpu
@pytest.mark.parametrize("io,b,D,strided", [("bf16", 1, 1, False), ("bf16", 3, 66, True), ("f32", 5, 40, False),
                                            ("f32", 2, 37, True), ("bf16", 130, 264, False)])
def test_forward_then_steps_equals_one_forward(io, b, D, strided):
    T0, K = 70, 5
    p = make(b, T0 + K, D, io, strided=strided, seed=b + D)
    ref = ref_of(p)
    cut = {k: p[k][:, :T0].contiguous() for k in ("x", "r", "i")}
    _, state = ssd.ssd_glr_fwd(cut["x"], cut["r"], cut["i"], p["A_log"], initial_states=p["init"],
                               return_final_states=True)
    for t in range(T0, T0 + K):
        y = ssd.ssd_glr_step(p["x"][:, t], p["r"][:, t], p["i"][:, t], p["A_log"], state)
        assert_within(f"token {t}", y, ref.h[:, t], ref.eh[:, t])
    assert_within("state", state, ref.final, ref.efinal)


# ------------------------------------------------------------------ GPU: use

@gpu
def test_a_malformed_cu_seqlens_is_reported_and_stays_in_bounds():
    for cu in ([0, 50, 40, 120], [5, 50, 80, 120], [0, 50, 80, 119], [0, -7, 3000, 120]):
        p = make(1, 120, 16, "bf16", cu=[0, 40, 80, 120])
        p["cu_t"] = torch.tensor(cu, dtype=torch.int32, device="cuda")
        for call in (fwd, bwd):
            with pytest.raises(ssd.SsdError) as e:
                call(p)
            assert e.value.code == -5
    check(make(1, 120, 16, "bf16", cu=[0, 40, 80, 120]))


@gpu
def test_outputs_stop_at_their_ends_and_the_workspace_may_be_dirty():
    p = make(1, 333, 37, "bf16", cu=[0, 100, 333], seed=8)
    want = fwd(p)
    buf = torch.full((400 * 37,), 7.0, dtype=torch.bfloat16, device="cuda")
    y = buf[:333 * 37].view(1, 333, 37)
    ws = torch.full((1 << 22,), 0xFF, dtype=torch.uint8, device="cuda")
    got = fwd(p, y=y, workspace=ws)
    assert all(torch.equal(a, b) for a, b in zip(got, want)) and bool((buf[333 * 37:] == 7.0).all())
    ws.fill_(0xFF)
    a, b = bwd(p), bwd(p, workspace=ws)
    assert all(torch.equal(a[k], b[k]) for k in a)


@gpu
def test_the_same_call_gives_the_same_bits_on_any_stream_and_in_a_graph():
    p = make(2, 3000, 200, "bf16", seed=9)
    y0, f0, c0 = fwd(p)
    g0 = bwd(p, chunk_states=c0)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    outs = []
    for s in streams:                                  # two calls at once, each with a workspace of its own
        with torch.cuda.stream(s):
            for _ in range(3):
                y, f, c = ssd.ssd_glr_fwd(p["x"], p["r"], p["i"], p["A_log"], initial_states=p["init"],
                                          return_final_states=True, return_chunk_states=True)
                g = ssd.ssd_glr_bwd(p["x"], p["r"], p["i"], p["A_log"], p["dy"], initial_states=p["init"],
                                    dfinal_states=p["dfinal"], chunk_states=c)
                outs.append((y, f, c, g))
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y, f, c = ssd.ssd_glr_fwd(p["x"], p["r"], p["i"], p["A_log"], initial_states=p["init"],
                                  return_final_states=True, return_chunk_states=True)
        g = ssd.ssd_glr_bwd(p["x"], p["r"], p["i"], p["A_log"], p["dy"], initial_states=p["init"],
                            dfinal_states=p["dfinal"])
    for _ in range(3):
        y.zero_(), f.zero_()
        graph.replay()
        torch.cuda.synchronize()
        outs.append((y, f, c, g))
    for y, f, c, g in outs:
        assert torch.equal(y, y0) and torch.equal(f, f0) and torch.equal(c, c0)
        assert all(torch.equal(g[k], g0[k]) for k in g0)


@gpu
def test_outputs_that_are_asked_for():
    p = make(2, 100, 16, "f32")
    args = (p["x"], p["r"], p["i"], p["A_log"])
    assert torch.is_tensor(ssd.ssd_glr_fwd(*args))
    y, c = ssd.ssd_glr_fwd(*args, return_chunk_states=True)
    assert c.shape == (2, 2, 16)
    f = torch.empty(2, 16, device="cuda")
    y, f2 = ssd.ssd_glr_fwd(*args, final_states=f)
    assert f2 is f
    assert ssd.ssd_glr_bwd(*args, p["dy"], want_dinitial=False)["dinitial_states"] is None
    with pytest.raises(ValueError):
        ssd.ssd_glr_bwd(*args, None)
