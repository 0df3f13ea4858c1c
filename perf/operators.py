"""Measured cases of the gated linear recurrence and the layer norm.

Each case is one call (or a forward and its backward) at sizes that the layer
meets: training batches and long rows of the widths of the benchmark's
workloads, packed batches, decoding batches of one to some hundred rows, odd
sizes.  `run` computes a case in plain torch operations (own = False) or
through the package's entry points (own = True).
"""
import math
import random

import torch
import torch.nn.functional as F

own = False

CHUNK = 64      # tokens between two kept states of the recurrence
LARGEST = 8 * 2048 * 5120

_T = {"bf16": torch.bfloat16, "f32": torch.float32}


def listed():
    return [
        # one token of one request (the 24-head, 64-channel layer's width): launch latency
        dict(name="step_1x1536_bf16", op="step", rows=1, dim=1536, dtype="bf16", fused=False),
        # one token of a decoding batch at the 80-head, 64-channel layer's width, gates cut from one projection
        dict(name="step_256x5120_bf16", op="step", rows=256, dim=5120, dtype="bf16", fused=True),
        # prefill of a batch of 2048-token rows, final states kept for decoding, gates cut from one projection
        dict(name="scan_8x2048x5120_bf16", op="scan", batch=8, tokens=2048, dim=5120, nseq=0, dtype="bf16", states=True,
             fused=True),
        # one long row: few channels for the GPU, so the time axis has to be split
        dict(name="scan_1x16384x2048_bf16", op="scan", batch=1, tokens=16384, dim=2048, nseq=0, dtype="bf16",
             states=True, fused=False),
        # packed sequences with entering states, float32
        dict(name="scan_packed_32768x1536_f32", op="scan", batch=1, tokens=32768, dim=1536, nseq=16, dtype="f32",
             states=True, fused=False),
        # a training step of the layer: forward and backward
        dict(name="train_8x2048x5120_bf16", op="train", batch=8, tokens=2048, dim=5120, nseq=0, dtype="bf16",
             states=False, fused=False, grads="io"),
        # backward of a small packed batch of ragged, empty and one-token sequences, odd width, nothing kept
        dict(name="scan_bwd_packed_5003x1030_f32", op="scan_bwd", batch=1, tokens=5003, dim=1030, nseq=9, dtype="f32",
             states=True, fused=True, grads="f32"),
        # pre-norm of a decoding batch, the residual stream carried along
        dict(name="norm_64x2560_bf16", op="norm", rows=64, dim=2560, groups=1, gate=False, residual=True, dtype="bf16"),
        # pre-norm of a training batch, statistics kept for the backward
        dict(name="norm_16384x5120_bf16", op="norm", rows=16384, dim=5120, groups=1, gate=False, residual=True,
             dtype="bf16"),
        # its backward, the residual stream's gradient added
        dict(name="norm_bwd_16384x5120_bf16", op="norm_bwd", rows=16384, dim=5120, groups=1, gate=False, residual=True,
             dtype="bf16", grads="io"),
        # the block's output norm, one group a head: forward and backward
        dict(name="gated_norm_16384x5120_bf16", op="norm", rows=16384, dim=5120, groups=80, gate=True, residual=False,
             dtype="bf16"),
        dict(name="gated_norm_bwd_32761x1536_bf16", op="norm_bwd", rows=32761, dim=1536, groups=24, gate=True,
             residual=False, dtype="bf16", grads="f32"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _width(rng, lo, hi):
    d = _log(rng, lo, hi)
    return d if rng.random() < 0.35 else max(8, d // 8 * 8)


def draw(rng):
    op = rng.choice(["step", "scan", "scan", "train", "scan_bwd", "norm", "norm", "norm_bwd", "norm_bwd"])
    dtype = rng.choice(["bf16", "bf16", "f32"])
    most = LARGEST // (2 if dtype == "f32" else 1) // (2 if op in ("train", "scan_bwd", "norm_bwd") else 1)
    if op == "step":
        return dict(op=op, rows=_log(rng, 1, 512), dim=_width(rng, 64, 8192), dtype=dtype, fused=rng.random() < 0.5)
    if op in ("norm", "norm_bwd"):
        gate = rng.random() < 0.4
        if gate:
            per, groups = rng.choice([32, 64, 64, 96, 128, 256, 61]), rng.randint(1, 96)
            dim = per * groups
        else:
            dim, groups = _width(rng, 64, 8192), 1
        rows = min(_log(rng, 1, 32768), max(1, most // dim))
        c = dict(op=op, rows=rows, dim=dim, groups=groups, gate=gate, residual=not gate and rng.random() < 0.6,
                 dtype=dtype)
        return dict(c, grads=rng.choice(["io", "f32"])) if op == "norm_bwd" else c
    dim = _width(rng, 64, 6144)
    tokens = min(_log(rng, 1, 32768), max(1, most // dim))
    nseq = rng.choice([0, 0, rng.randint(1, 24)])
    batch = 1 if nseq else max(1, min(_log(rng, 1, 16), most // dim // tokens))
    c = dict(op=op, batch=batch, tokens=tokens, dim=dim, nseq=nseq, dtype=dtype, states=rng.random() < 0.6,
             fused=rng.random() < 0.5)
    return c if op == "scan" else dict(c, grads=rng.choice(["io", "f32"]))


def _lengths(case):
    """Lengths of a packed batch: ragged, now and then empty or of one token."""
    n, T = case["nseq"], case["tokens"]
    rng = random.Random(1000003 * T + n)
    cuts = sorted(rng.randint(0, T) for _ in range(n - 1))
    if len(cuts) >= 4:
        cuts[1] = cuts[0]                         # an empty sequence
        cuts[3] = min(cuts[2] + 1, T)             # one of a single token
        cuts = sorted(cuts)
    edges = [0] + cuts + [T]
    return [b - a for a, b in zip(edges, edges[1:])]


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    io = _T[case["dtype"]]

    def normal(*shape, std=1.0, mean=0.0):
        return torch.randn(shape, generator=gen, device="cuda", dtype=torch.float32).mul_(std).add_(mean)

    s = dict(case)
    if case["op"] in ("norm", "norm_bwd"):
        R, D, G = case["rows"], case["dim"], case["groups"]
        s["x"] = normal(R, D, mean=0.1).to(io)
        s["weight"], s["bias"] = normal(D, std=0.1, mean=1.0), normal(D, std=0.1)
        s["z"] = normal(R, D).to(io) if case["gate"] else None
        s["res"] = normal(R, D).to(io) if case["residual"] else None
        if case["op"] == "norm_bwd":
            gdt = io if case["grads"] == "io" else torch.float32
            s["gdt"] = gdt
            s["dy"] = normal(R, D).to(io)
            s["res"] = None
            s["dres"] = normal(R, D).to(gdt) if case["residual"] else None
            u = s["x"].double()
            u = (u * s["z"].double() * torch.sigmoid(s["z"].double()) if case["gate"] else u).view(R, G, D // G)
            s["mean"] = u.mean(2).float()
            s["rstd"] = (u.var(2, unbiased=False) + 1e-5).rsqrt().float()
        return s
    if case["op"] == "step":
        lead, nstate = (case["rows"],), case["rows"]
    else:
        lead, nstate = (case["batch"], case["tokens"]), case["nseq"] or case["batch"]
    D = case["dim"]
    if case["fused"]:                             # x and the gates are thirds of one projection's output
        s["x"], s["r"], s["i"] = normal(*lead, 3 * D).to(io).split(D, dim=-1)
    else:
        s["x"], s["r"], s["i"] = (normal(*lead, D).to(io) for _ in range(3))
    # rates that leave 0.43 to 0.992 of the state a token where the gate is open
    s["A_log"] = torch.rand(D, generator=gen, device="cuda") * 4.6 - 4.8
    if case["op"] == "step":
        s["state"] = normal(nstate, D)
        return s
    s["init"] = normal(nstate, D, std=0.5) if case["states"] else None
    s["cu"] = s["first"] = s["last"] = s["full"] = None
    if case["nseq"]:
        lens = _lengths(case)
        cu = torch.tensor([0] + lens, dtype=torch.int64).cumsum(0)
        keep = torch.tensor([k for k, n in enumerate(lens) if n], dtype=torch.int64)
        s["cu"] = cu.to(torch.int32).cuda()
        s["full"] = keep.cuda()                   # sequences that have tokens, their first and last tokens
        s["first"], s["last"] = cu[:-1][keep].cuda(), cu[1:][keep].cuda() - 1
    if case["op"] != "scan":
        s["gdt"] = io if case["grads"] == "io" else torch.float32
        s["dy"] = normal(*lead, D).to(io)
        s["dfinal"] = normal(nstate, D) if case["states"] else None
    return s


# ------------------------------------------------------------------ plain forms

def _gates(s):
    r, i = s["r"].float(), s["i"].float()
    sr, si = 1 / (1 + torch.exp(-r)), 1 / (1 + torch.exp(-i))
    q = torch.exp(s["A_log"]) * sr
    e = torch.expm1(-q)                           # a - 1
    return sr, si, q, torch.exp(-q), torch.sqrt(-e * (2 + e))


def _recur(a, b):
    """h_t = a_t h_{t-1} + b_t along dim 1 from h = 0: pairs are joined, the half as long row solved, and filled in."""
    if a.shape[1] <= 1:
        return b
    n = a.shape[1] // 2
    ae, be, ao, bo = a[:, 0:2 * n:2], b[:, 0:2 * n:2], a[:, 1::2], b[:, 1::2]
    odd = _recur(ao * ae, torch.addcmul(bo, ao, be))
    h = torch.empty_like(b)
    h[:, 1::2] = odd
    h[:, 0] = b[:, 0]
    h[:, 2::2] = torch.addcmul(b[:, 2::2], a[:, 2::2], odd[:, : (a.shape[1] - 1) // 2])
    return h


def _plain_states(s, a, b):
    """States h in 32 bits, the states before each token, and the final states."""
    T, init = a.shape[1], s["init"]
    if s["cu"] is None:
        start = torch.zeros_like(b[:, 0]) if init is None else init
        b = torch.cat([torch.addcmul(b[:, :1], a[:, :1], start[:, None]), b[:, 1:]], 1)
        h = _recur(a, b)
        return h, torch.cat([start[:, None], h[:, :-1]], 1), h[:, T - 1].clone()
    first, last, full = s["first"], s["last"], s["full"]
    start = torch.zeros((s["nseq"], a.shape[2]), device=a.device) if init is None else init
    b = b.clone()
    b[0, first] = torch.addcmul(b[0, first], a[0, first], start[full])
    a = a.clone()
    a[0, first] = 0
    h = _recur(a, b)
    before = torch.cat([h[:, :1], h[:, :-1]], 1)
    before[0, first] = start[full]
    final = start.clone()
    final[full] = h[0, last]
    return h, before, final


def _plain_scan(s):
    sr, si, q, a, m = _gates(s)
    h, before, final = _plain_states(s, a, m * si * s["x"].float())
    return h.to(s["x"].dtype), final


def _plain_scan_bwd(s, before=None):
    sr, si, q, a, m = _gates(s)
    x, dy = s["x"].float(), s["dy"].float()
    if before is None:
        before = _plain_states(s, a, m * si * x)[1]
    nxt = torch.cat([a[:, 1:], torch.zeros_like(a[:, :1])], 1)
    if s["cu"] is None:
        if s["dfinal"] is not None:
            dy = torch.cat([dy[:, :-1], dy[:, -1:] + s["dfinal"][:, None]], 1)
    else:
        nxt[0, s["last"]] = 0
        dy = dy.clone()
        if s["dfinal"] is not None:
            dy[0, s["last"]] += s["dfinal"][s["full"]]
    g = _recur(nxt.flip(1), dy.flip(1)).flip(1)
    if s["cu"] is None:
        dinit = a[:, 0] * g[:, 0]
    else:
        dinit = torch.zeros((s["nseq"], a.shape[2]), device=a.device) if s["dfinal"] is None else s["dfinal"].clone()
        dinit[s["full"]] = a[0, s["first"]] * g[0, s["first"]]
    gsx = g * si * x
    dq = a * (a / m * gsx - g * before)
    gdt = s["gdt"]
    return dict(dx=(g * m * si).to(gdt), dr=(dq * q * (1 - sr)).to(gdt), di=(m * gsx * (1 - si)).to(gdt),
                dA_log=(dq * q).sum((0, 1)), dinitial_states=dinit)


def _plain_train(s):
    sr, si, q, a, m = _gates(s)
    h, before, final = _plain_states(s, a, m * si * s["x"].float())
    return dict(_plain_scan_bwd(s, before), y=h.to(s["x"].dtype))


def _plain_step(s):
    sr, si, q, a, m = _gates(s)
    s["state"].mul_(a).add_(m * si * s["x"].float())
    return s["state"].to(s["x"].dtype), s["state"]


def _plain_norm(s):
    x, R, G = s["x"], s["rows"], s["groups"]
    u, total = x.float(), None
    if s["res"] is not None:
        total = (u + s["res"].float()).to(x.dtype)    # what is normalised is the sum that is kept
        u = total.float()
    if s["z"] is not None:
        z = s["z"].float()
        u = u * (z / (1 + torch.exp(-z)))
    u = u.view(R, G, -1)
    mean = u.mean(2, keepdim=True)
    c = u - mean
    rstd = 1 / torch.sqrt((c * c).mean(2, keepdim=True) + 1e-5)
    y = (c * rstd).view(R, -1) * s["weight"] + s["bias"]
    return dict(y=y.to(x.dtype), total=total, mean=mean.view(R, G), rstd=rstd.view(R, G))


def _plain_norm_bwd(s):
    R, G = s["rows"], s["groups"]
    x, dy, z = s["x"].float(), s["dy"].float(), s["z"]
    gate = None
    if z is not None:
        z = z.float()
        sz = 1 / (1 + torch.exp(-z))
        gate = z * sz
    mean, rstd = s["mean"].view(R, G, 1), s["rstd"].view(R, G, 1)
    xh = ((x if gate is None else x * gate).view(R, G, -1) - mean) * rstd
    wdy = (dy * s["weight"]).view(R, G, -1)
    du = rstd * (wdy - wdy.mean(2, keepdim=True) - xh * (wdy * xh).mean(2, keepdim=True))
    du, xh, gdt, dz = du.view(R, -1), xh.view(R, -1), s["gdt"], None
    if gate is not None:
        dz = (du * x * sz * (1 + z * (1 - sz))).to(gdt)
        du = du * gate
    if s["dres"] is not None:
        du = du + s["dres"].float()
    return dict(dx=du.to(gdt), dz=dz, dweight=(dy * xh).sum(0), dbias=dy.sum(0))


# ------------------------------------------------------------------ the package's calls

def _own(s):
    import mamba_ssd_layer_fwd_b200 as ssd
    op = s["op"]
    if op == "step":
        return ssd.ssd_glr_step(s["x"], s["r"], s["i"], s["A_log"], s["state"]), s["state"]
    if op == "scan":
        return ssd.ssd_glr_fwd(s["x"], s["r"], s["i"], s["A_log"], initial_states=s["init"], cu_seqlens=s["cu"],
                               return_final_states=True)
    if op == "train":
        y, kept = ssd.ssd_glr_fwd(s["x"], s["r"], s["i"], s["A_log"], initial_states=s["init"], cu_seqlens=s["cu"],
                                  return_chunk_states=True)
        return dict(ssd.ssd_glr_bwd(s["x"], s["r"], s["i"], s["A_log"], s["dy"], initial_states=s["init"],
                                    cu_seqlens=s["cu"], dfinal_states=s["dfinal"], chunk_states=kept,
                                    grad_dtype=s["gdt"]), y=y)
    if op == "scan_bwd":
        return ssd.ssd_glr_bwd(s["x"], s["r"], s["i"], s["A_log"], s["dy"], initial_states=s["init"],
                               cu_seqlens=s["cu"], dfinal_states=s["dfinal"], grad_dtype=s["gdt"])
    if op == "norm":
        out = ssd.ssd_layer_norm_fwd(s["x"], s["weight"], s["bias"], residual=s["res"], z=s["z"], ngroups=s["groups"],
                                     eps=1e-5, return_stats=True)
        if s["res"] is None:
            return dict(y=out[0], total=None, mean=out[1], rstd=out[2])
        return dict(y=out[0], total=out[1], mean=out[2], rstd=out[3])
    return ssd.ssd_layer_norm_bwd(s["x"], s["weight"], s["dy"], s["mean"], s["rstd"], z=s["z"], dresidual=s["dres"],
                                  ngroups=s["groups"], grad_dtype=s["gdt"])


def run(state):
    if own:
        return _own(state)
    return {"step": _plain_step, "scan": _plain_scan, "train": _plain_train, "scan_bwd": _plain_scan_bwd,
            "norm": _plain_norm, "norm_bwd": _plain_norm_bwd}[state["op"]](state)


def work(case):
    b = 2 if case["dtype"] == "bf16" else 4
    g = b if case.get("grads") == "io" else 4
    D = case["dim"]
    if case["op"] == "step":
        n = case["rows"] * D
        return dict(bytes=n * (4 * b + 8) + 4 * D, flops=20 * n)
    if case["op"] in ("norm", "norm_bwd"):
        n, st = case["rows"] * D, 8 * case["rows"] * case["groups"]
        if case["op"] == "norm":
            return dict(bytes=n * b * (2 + case["gate"] + 2 * case["residual"]) + st + 8 * D,
                        flops=n * (8 + 5 * case["gate"]))
        return dict(bytes=n * (b * (2 + case["gate"]) + g * (1 + case["gate"] + case["residual"])) + st + 12 * D,
                    flops=n * (14 + 10 * case["gate"]))
    n = case["batch"] * case["tokens"] * D
    st = 4 * D * (case["nseq"] or case["batch"])
    if case["op"] == "scan":
        return dict(bytes=n * 4 * b + st * (1 + case["states"]) + 4 * D, flops=20 * n)
    if case["op"] == "scan_bwd":
        return dict(bytes=n * (4 * b + 3 * g) + st * (1 + 2 * case["states"]) + 8 * D, flops=45 * n)
    # forward and backward: x, r and i are read in each, beside y, dy and the gradients
    return dict(bytes=n * (8 * b + 3 * g) + st * (1 + 3 * case["states"]) + 12 * D, flops=65 * n)


# ------------------------------------------------------------------ the definition, in 64 bits

def exact(case, seed):
    s = prepare(case, seed)
    x = s["x"].double()
    if case["op"] in ("norm", "norm_bwd"):
        return _exact_norm(s, x)
    r, i = s["r"].double(), s["i"].double()
    rate = s["A_log"].double().exp()
    a = torch.exp(-rate * torch.sigmoid(r))
    m = torch.sqrt(-torch.expm1(-2 * rate * torch.sigmoid(r)))
    si = torch.sigmoid(i)
    if case["op"] == "step":
        h = a * s["state"].double() + m * si * x
        return h, h
    spans = [(0, case["tokens"])]
    if case["nseq"]:
        edges = s["cu"].tolist()
        spans = list(zip(edges, edges[1:]))
    nstate = case["nseq"] or case["batch"]
    start = torch.zeros((nstate, case["dim"]), device="cuda", dtype=torch.float64)
    if s["init"] is not None:
        start = s["init"].double()
    h, before, final = torch.empty_like(x), torch.empty_like(x), start.clone()
    b = m * si * x
    for k, (lo, hi) in enumerate(spans):
        c = start[k:k + 1] if case["nseq"] else start
        for t in range(lo, hi):
            before[:, t] = c
            c = torch.addcmul(b[:, t], a[:, t], c)
            h[:, t] = c
        if case["nseq"]:
            final[k] = c[0]
        else:
            final = c
    if case["op"] == "scan":
        return h, final
    del b
    dy, g, dinit = s["dy"].double(), torch.empty_like(x), torch.empty_like(start)
    end = torch.zeros_like(start) if s["dfinal"] is None else s["dfinal"].double()
    for k, (lo, hi) in enumerate(spans):
        c = end[k:k + 1] if case["nseq"] else end
        for t in range(hi - 1, lo - 1, -1):
            g[:, t] = dy[:, t] + c
            c = a[:, t] * g[:, t]
        if case["nseq"]:
            dinit[k] = c[0]
        else:
            dinit = c
    dq = g * (a * a / m * si * x - a * before)
    q = rate * torch.sigmoid(r)
    out = dict(dx=g * m * si, dr=dq * q * torch.sigmoid(-r), di=g * m * x * si * torch.sigmoid(-i),
               dA_log=(dq * q).sum((0, 1)), dinitial_states=dinit)
    return dict(out, y=h) if case["op"] == "train" else out


def _exact_norm(s, x):
    R, G = s["rows"], s["groups"]
    w, total = s["weight"].double(), None
    if s["res"] is not None:
        total = x + s["res"].double()
        x = total.to(s["x"].dtype).double()
    u = x if s["z"] is None else x * F.silu(s["z"].double())
    u = u.view(R, G, -1)
    if s["op"] == "norm":
        rstd = (u.var(2, unbiased=False) + 1e-5).rsqrt()
        hat = ((u - u.mean(2, keepdim=True)) * rstd[..., None]).view(R, -1)
        return dict(y=hat * w + s["bias"].double(), total=total, mean=u.mean(2), rstd=rstd)
    mean, rstd, dy = s["mean"].double(), s["rstd"].double(), s["dy"].double()
    hat = (u - mean[..., None]) * rstd[..., None]
    wd = (dy * w).view(R, G, -1)
    P = wd.shape[2]
    du = wd - (wd.sum(2, keepdim=True) + hat * (wd * hat).sum(2, keepdim=True)) / P
    du = (du * rstd[..., None]).view(R, -1)
    dz = None
    if s["z"] is not None:
        z = s["z"].double()
        sg = torch.sigmoid(z)
        dz, du = du * x * (sg + z * sg * (1 - sg)), du * F.silu(z)
    if s["dres"] is not None:
        du = du + s["dres"].double()
    return dict(dx=du, dz=dz, dweight=(dy * hat.view(R, -1)).sum(0), dbias=dy.sum(0))
