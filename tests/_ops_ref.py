"""Plain 64-bit forms of the gated linear recurrence and the layer norm, with
bounds on what float32 arithmetic may add, for the operators' tests.

Every bound is a first-order running error analysis in U = 2^-24 (half a step
of float32, relative).  Outputs in bf16 may be off by half a step of bf16 more:
`tol` adds 2^-8 of the value."""
import torch

U = 2.0 ** -24
# The kernels take q + 2^-124 for q, so that m = sqrt(1 - a^2) is above 0 and 1 / m finite: 1 - a^2 = 1 - exp(-2 q) is
# off by at most 2^-123, its root by at most 2^-61.5, which is what is left of it at q = 0.  The gradient's q a^2 / m,
# which goes as sqrt(q / 2) there, is off by at most sqrt(2^-125) = 2^-62.5.
M0 = 2.0 ** -61


def half_step(dtype) -> float:
    return torch.finfo(dtype).eps / 2


def tol(value, err, dtype):
    """Largest difference allowed for an output of `dtype`: err before rounding, half a step after."""
    return err + half_step(dtype) * (value.abs() + err) + 1e-30


def assert_within(name, got, value, err):
    assert got.shape == value.shape, (name, tuple(got.shape), tuple(value.shape))
    if got.numel() == 0:
        return
    g = got.double().to(value.device)
    assert bool(torch.isfinite(g).all()), f"{name}: non-finite values"
    d, t = (g - value).abs(), tol(value, err, got.dtype)
    worst = float((d / t).max())
    assert worst <= 1.0, f"{name}: {worst:.3g} times its bound (max |d| {float(d.max()):.3e})"


def spans_of(b, T, cu=None):
    """[(row, first token, end, state index)]"""
    if cu is None:
        return [(k, 0, T, k) for k in range(b)]
    return [(0, lo, hi, k) for k, (lo, hi) in enumerate(zip(cu, cu[1:]))]


class Glr:
    """The recurrence in 64 bits: y (before rounding), final states, chunk
    states, and `grad`; `e_*` are the bounds.  x, r, i (b, T, D)."""

    def __init__(self, x, r, i, A_log, init=None, cu=None, chunk=64):
        dev = x.device
        x, r, i = x.double(), r.double(), i.double()
        b, T, D = x.shape
        self.x, self.r, self.i = x, r, i
        rate = A_log.double().exp().to(dev)
        self.sr, self.si = torch.sigmoid(r), torch.sigmoid(i)
        self.osr, self.osi = torch.sigmoid(-r), torch.sigmoid(-i)
        q = self.q = rate * self.sr
        self.a, self.m = torch.exp(-q), torch.sqrt(-torch.expm1(-2 * q))
        # sigmoid: exponent's argument off by 2U|r|, exp by 4U, sums and products by some U; the shared
        # reciprocal brings in the other gate's rounding too
        big = max([1.0] + [float(v.abs().clamp(max=64).max()) for v in (r, i) if v.numel()])
        self.ds = ds = (16 + 4 * big) * U
        self.dq = ds + 8 * U                              # q: times exp(A_log), itself within 4U
        self.da = 8 * U + q.clamp(max=90) * self.dq       # a = exp(-q)
        self.db = self.dq + ds + 16 * U                   # m sigmoid(i) x: m is off by at most what q is
        self.spans = spans_of(b, T, cu)
        nstate = len(self.spans)
        init = torch.zeros((nstate, D), dtype=torch.float64, device=dev) if init is None else init.double().to(dev)
        self.h, self.before = torch.zeros_like(x), torch.zeros_like(x)
        self.eh, self.ebefore = torch.zeros_like(x), torch.zeros_like(x)
        self.final, self.efinal = init.clone(), torch.zeros_like(init)
        bt = self.m * self.si * x
        m0 = 2 * M0 * (self.si * x).abs()
        for row, lo, hi, k in self.spans:
            h, H, E = init[k], init[k].abs(), torch.zeros_like(init[k])
            for t in range(lo, hi):
                a = self.a[row, t]
                self.before[row, t], self.ebefore[row, t] = h, E + 16 * U * H
                E = a * E + (self.da[row, t] + 4 * U) * a * H + self.db * bt[row, t].abs() + m0[row, t]
                h, H = a * h + bt[row, t], a * H + bt[row, t].abs()
                E = E + 2 * U * H
                self.h[row, t], self.eh[row, t] = h, E + 16 * U * H
            self.final[k], self.efinal[k] = h, E + (16 * U * H if hi > lo else 0)
        self.chunks, self.echunks = self.before[:, ::chunk], self.ebefore[:, ::chunk]

    def grad(self, dy, dfinal=None):
        """{name: (value, bound)}"""
        x, a, m, q, si = self.x, self.a, self.m, self.q, self.si
        dy = dy.double()
        dinit = torch.zeros_like(self.final) if dfinal is None else dfinal.double().to(x.device).clone()
        edinit = torch.zeros_like(dinit)
        g, eg = torch.zeros_like(x), torch.zeros_like(x)
        for row, lo, hi, k in self.spans:
            c, C, E = dinit[k].clone(), dinit[k].abs(), torch.zeros_like(dinit[k])
            for t in range(hi - 1, lo - 1, -1):
                g[row, t], G = dy[row, t] + c, dy[row, t].abs() + C
                eg[row, t] = E + 16 * U * G
                c, C = a[row, t] * g[row, t], a[row, t] * G
                E = a[row, t] * (E + 2 * U * G) + (self.da[row, t] + 4 * U) * C
            dinit[k], edinit[k] = c, E + (16 * U * C if hi > lo else 0)
        ag, ax = g.abs(), x.abs()
        k1 = torch.where(m > 0, q * a * a / m.clamp(min=1e-300), torch.zeros_like(m)) * si * ax
        k2 = q * a
        dqq = torch.where(m > 0, q * a * a / m.clamp(min=1e-300), torch.zeros_like(m)) * si * x * g - k2 * g * self.before
        e = k1 * (eg + ag * (3 * self.dq + 2 * self.da + self.ds + 32 * U))
        e = e + k2 * (eg * self.before.abs() + ag * self.ebefore
                      + ag * self.before.abs() * (self.dq + self.da + 16 * U))
        e = e + 2 * M0 * si * ax * ag + 2.0 ** -123 * ag * self.before.abs()
        return {
            "dx": (g * m * si, m * si * (eg + ag * (self.db + 8 * U)) + 2 * M0 * si * ag),
            "di": (g * m * x * si * self.osi, (m * (eg + ag * (self.db + self.ds + 16 * U)) + 2 * M0 * ag) * si * self.osi * ax),
            "dr": (dqq * self.osr, self.osr * (e + dqq.abs() * (self.ds + 8 * U))),
            "dA_log": (dqq.sum((0, 1)), (e + 256 * U * dqq.abs()).sum((0, 1))),
            "dinitial_states": (dinit, edinit),
        }


class Norm:
    """The layer norm in 64 bits.  x, z, res (..., D)."""

    def __init__(self, x, weight, bias=None, res=None, z=None, groups=1, eps=1e-5):
        D = x.shape[-1]
        self.shape, self.G, self.z = x.shape, groups, None
        self.w = weight.double().to(x.device)
        b = torch.zeros_like(self.w) if bias is None else bias.double().to(x.device)
        self.x = x.double()
        self.total = None
        if res is not None:
            self.total = self.x + res.double()
            self.x = (x.float() + res.float()).to(x.dtype).double()
        u, eu = self.x, torch.zeros_like(self.x)
        if z is not None:
            self.z = z.double()
            self.dz_rel = (16 + 4 * float(self.z.abs().max() if z.numel() else 0)) * U   # silu, its slope
            u = u * self.z * torch.sigmoid(self.z)
            eu = self.dz_rel * u.abs()
        self.u, self.eu = self._split(u), self._split(eu)
        self.mean = self.u.mean(-1, keepdim=True)
        em = self.eu.mean(-1, keepdim=True) + 64 * U * self.u.abs().mean(-1, keepdim=True)
        self.emean = em
        c = self.u - self.mean
        ec = em + self.eu + 2 * U * (self.u.abs() + self.mean.abs())
        var = (c * c).mean(-1, keepdim=True)
        evar = (2 * c.abs() * ec + ec * ec).mean(-1, keepdim=True) + 64 * U * var
        self.rstd = (var + eps).rsqrt()
        rel = 0.5 * evar / (var + eps) + 8 * U
        self.erstd = self.rstd * rel
        hat = c * self.rstd
        ehat = self.rstd * ec * (1 + rel) + hat.abs() * (rel + 4 * U)
        w, bb = self._split(self.w.expand(x.shape)), self._split(b.expand(x.shape))
        self.y = (hat * w + bb).reshape(x.shape)
        self.ey = (ehat * w.abs() + 4 * U * ((hat * w).abs() + bb.abs())).reshape(x.shape)

    def _split(self, v):
        return v.reshape(self.shape[:-1] + (self.G, self.shape[-1] // self.G))

    def stats(self):
        return self.mean[..., 0], self.rstd[..., 0]

    def grad(self, dy, mean, rstd, dres=None):
        """{name: (value, bound)} for the float32 statistics given."""
        mean, rstd = mean.double().unsqueeze(-1), rstd.double().unsqueeze(-1)
        dy_ = self._split(dy.double())
        w = self._split(self.w.expand(self.shape))
        xh = (self.u - mean) * rstd
        exh = rstd * (self.eu + 2 * U * (self.u.abs() + mean.abs())) + 4 * U * xh.abs()
        wd = dy_ * w
        s1, s2 = wd.mean(-1, keepdim=True), (wd * xh).mean(-1, keepdim=True)
        es1 = 64 * U * wd.abs().mean(-1, keepdim=True)
        es2 = (wd.abs() * exh).mean(-1, keepdim=True) + 64 * U * (wd * xh).abs().mean(-1, keepdim=True)
        du = rstd * (wd - s1 - xh * s2)
        edu = rstd * (8 * U * (wd.abs() + s1.abs() + (xh * s2).abs()) + es1 + xh.abs() * es2 + s2.abs() * exh)
        du, edu = du.reshape(self.shape), edu.reshape(self.shape)
        lead = tuple(range(len(self.shape) - 1))
        flat = lambda v: v.reshape(self.shape)
        out = {"dweight": (flat(dy_ * xh).sum(lead), flat(dy_.abs() * exh + 256 * U * (dy_ * xh).abs()).sum(lead)),
               "dbias": (flat(dy_).sum(lead), 256 * U * flat(dy_).abs().sum(lead))}
        if self.z is None:
            v = du if dres is None else du + dres.double()
            return dict(out, dx=(v, edu + 2 * U * v.abs()))
        s = torch.sigmoid(self.z)
        gate, slope = self.z * s, s * (1 + self.z * (1 - s))
        rel = self.dz_rel + 8 * U
        # the slope's two terms cancel near its zero: its error goes with their absolute values
        slope_abs = s * (1 + self.z.abs() * (1 - s))
        return dict(out, dx=(du * gate, (edu + rel * du.abs()) * gate.abs()),
                    dz=(du * self.x * slope, self.x.abs() * (edu * slope.abs() + rel * du.abs() * slope_abs)))
