"""References of the norms and losses in binary64 (torch), from the definitions, and bounds of what binary32
arithmetic may be off.

A bound counts units of 2^-24 (half a step of binary32, relative) of the sum of the magnitudes that a value is
made of: n roundings in a row are off by at most n * 2^-24 of it to first order."""
import torch

U = 2.0 ** -24
HALF = {t: torch.finfo(t).eps / 2 for t in (torch.float32, torch.bfloat16, torch.float16)}
TINY = {torch.float32: 2.0 ** -149, torch.bfloat16: 2.0 ** -133, torch.float16: 2.0 ** -24}
EPS = 1e-5


def rounding(ref, dtype):
    """The rounding of a stored value: half a step, also below the normal numbers."""
    return HALF[dtype] * ref.abs() + TINY[dtype]


def check(got, ref, bound, what=""):
    """|got - ref| within the bound plus got's own rounding (of a value that may itself be off by the bound)."""
    assert got.shape == ref.shape, what
    d = (got.double() - ref).abs()
    ok = d <= bound + rounding(ref.abs() + bound, got.dtype)
    assert bool(ok.all()), (what, float((d / (bound + rounding(ref, got.dtype))).max()))


# ---------------------------------------------------------------- norms
def stats64(x, kind):
    mean = x.mean(1, keepdim=True) if kind == "layer" else torch.zeros_like(x[:, :1])
    return mean, 1.0 / torch.sqrt(((x - mean) ** 2).mean(1, keepdim=True) + EPS)


class Norm64:
    """The pass in binary64 on given h, r, r' (as stored), with magnitudes.

    Additions in a row: 8 of a thread, 5 in a warp, 4 or 5 over the warps and CTAs; a mean then has its factor,
    rstd its own sum, square root and reciprocal (2 units): below 32 in all for a normed value, twice that where a
    second mean follows."""

    def __init__(self, h, r, r_out, pre, post, w, b, post_w, post_b, gate, res_scale):
        f = lambda t: None if t is None else t.double()  # noqa: E731
        h, r, r_out, w, b, post_w, post_b, gate = map(f, (h, r, r_out, w, b, post_w, post_b, gate))
        rows, cols = r.shape
        one, zero = r.new_ones(cols), r.new_zeros(cols)
        self.w, self.b = one if w is None else w, zero if b is None else b
        self.pw, self.pb = one if post_w is None else post_w, zero if post_b is None else post_b
        self.gates = 1 if gate is None or gate.dim() == 1 else gate.shape[0]
        g = one if gate is None else gate
        self.g = g.view(-1, cols).repeat_interleave(rows // self.gates, 0) if rows else g.view(-1, cols)[:0]
        self.pre, self.post, self.alpha, self.r_out = pre, post, res_scale, r_out
        u, self.u_mag = (torch.zeros_like(r), torch.zeros_like(r)) if h is None else (h, h.abs())
        self.h = h
        if post != "none":
            self.mean1, self.rho1 = stats64(h, post)
            self.n1 = (h - self.mean1) * self.rho1
            # a mean of mixed signs is off by units of the mean magnitude
            self.n1_mag = (h.abs() + h.abs().mean(1, keepdim=True)) * self.rho1
            u, self.u_mag = self.n1 * self.pw + self.pb, self.n1_mag * self.pw.abs() + self.pb.abs()
        self.u = u
        self.r_new, self.r_mag = res_scale * r + self.g * u, abs(res_scale) * r.abs() + self.g.abs() * self.u_mag
        if pre != "none":
            self.mean2, self.rho2 = stats64(r_out, pre)
            self.n2 = (r_out - self.mean2) * self.rho2
            self.n2_mag = (r_out.abs() + r_out.abs().mean(1, keepdim=True)) * self.rho2
            self.x, self.x_mag = self.n2 * self.w + self.b, self.n2_mag * self.w.abs() + self.b.abs()

    @staticmethod
    def _back(dn, mag, n, n_mag, rho, kind):
        m = lambda t: t.mean(1, keepdim=True)  # noqa: E731
        d, a = dn - n * m(dn * n), mag + n_mag * m(mag * n_mag)
        if kind == "layer":
            d, a = d - m(dn), a + m(mag)
        return d * rho, a * rho

    def backward(self, dx, dr_out):
        """{name: (value, magnitude)}."""
        out = {}
        G = torch.zeros_like(self.r_out) if dr_out is None else dr_out.double()
        G_mag = G.abs()
        if self.pre != "none":
            dx = dx.double()
            d, a = self._back(dx * self.w, (dx * self.w).abs(), self.n2, self.n2_mag, self.rho2, self.pre)
            G, G_mag = G + d, G_mag + a
            out["dw"] = ((dx * self.n2).sum(0), (dx.abs() * self.n2_mag).sum(0))
            out["db"] = (dx.sum(0), dx.abs().sum(0))
        out["dr"] = (self.alpha * G, abs(self.alpha) * G_mag)
        if self.h is None:
            return out
        per = lambda t: t.view(self.gates, -1, t.shape[1]).sum(1)  # noqa: E731
        out["dgate"] = (per(G * self.u), per(G_mag * self.u_mag))
        du, du_mag = G * self.g, G_mag * self.g.abs()
        if self.post != "none":
            out["dpost_w"] = ((du * self.n1).sum(0), (du_mag * self.n1_mag).sum(0))
            out["dpost_b"] = (du.sum(0), du_mag.sum(0))
            du, du_mag = self._back(du * self.pw, du_mag * self.pw.abs(), self.n1, self.n1_mag, self.rho1, self.post)
        out["dh"] = (du, du_mag)
        return out


# ---------------------------------------------------------------- softmax losses
class Rows64:
    """softmax(beta z) of each row in binary64, with what binary32 may be off.

    An exponent's argument (z - m) beta log2 e has four roundings (two constants, two products), so e^a is off by
    4 |a| + 4 units (the function's own error is 2 units of 2^-23); a thread adds up `run` terms and then at most 24
    in the joins."""

    def __init__(self, z, beta, run):
        s = z.double() * beta
        self.none = torch.isneginf(s).all(1)
        m = torch.where(self.none, torch.zeros_like(s[:, 0]), s.amax(1))[:, None]
        a = s - m
        e = torch.exp(a)
        self.total = e.sum(1)
        self.log_total = torch.log(self.total)
        self.lp = a - self.log_total[:, None]
        self.p = torch.where(self.none[:, None], torch.zeros_like(e), e / self.total.clamp_min(1e-300)[:, None])
        self.a = torch.where(e > 0, a.abs(), torch.zeros_like(a))
        # relative error of the total, units
        self.total_units = (self.p * (4 * self.a + 4)).sum(1) + run + 24
        self.p_units = 4 * self.a + 8 + self.total_units[:, None]
        self.entropy = torch.special.entr(self.p).sum(1)

    def logp_bound(self, lp, a):
        total = self.total_units if lp.dim() == 1 else self.total_units[:, None]
        return U * (total + 4 * a + 4 * lp.abs() + 4)

    def entropy_bound(self):
        """log S - W / S: each term of W has the error of its e and of its argument."""
        w = (self.p * self.a * (4 * self.a + 8)).sum(1) + (self.p * self.a).sum(1) * (2 * self.total_units + 8)
        return U * (w + self.total_units + 4 * self.log_total.abs() + 4 * self.entropy.abs() + 4)
