"""Cross entropy gradients of up to 64 tokens in 16 bits.  A row's weight gradient is then a few
tokens' dz times their hidden states, so that a rounding of dz is as large as the gradient's own:
dz is held in two parts.

Tolerances, with u = 2^-24 and r, s the relative and absolute half steps of the type:
- dz is off by what the logit's error makes of p and by 4 u of p and of the target's 1; its two
  parts leave out r of r of it (f16: and s of the largest dloss / 2^13 for the smallest parts);
- a gradient is off by its terms' errors, by (n + 256) u of its n terms' sizes, and by r and s
  for its rounding.
"""
import torch

TYPES = {"f16": torch.float16, "bf16": torch.bfloat16}
U = 2.0 ** -24


class Few:
    def __init__(self, tokens, rows, cols, t, seed, device, pad=0, ignored=0):
        g = torch.Generator(device=device)
        g.manual_seed(seed)
        n = lambda *s: torch.randn(*s, generator=g, device=device)  # noqa: E731
        self.tokens, self.rows, self.cols, self.t, self.ld = tokens, rows, cols, t, cols + pad
        self.hidden = n(tokens, self.ld).to(TYPES[t])[:, :cols]
        self.weights = [(n(k, self.ld) * (2.0 / cols ** 0.5)).to(TYPES[t])[:, :cols] for k in rows]
        # all targets in the first shard: the others' gradients are p dloss h alone
        self.targets = torch.randint(0, rows[0], (tokens,), generator=g, device=device)
        self.targets[:ignored] = -100
        self.dloss = 0.5 + torch.rand(tokens, generator=g, device=device)
        self.h, self.w = self.hidden.double(), torch.cat(self.weights).double()
        z = self.h @ self.w.T
        self.lse = torch.logsumexp(z, 1).float()
        x = z - self.lse.double()[:, None]
        p = x.exp()
        self.scale = torch.where(self.targets >= 0, self.dloss.double(), 0.0)[:, None]
        self.hit = torch.zeros_like(p).scatter_(1, self.targets.clamp(min=0)[:, None], 1.0)
        self.dz = (p - self.hit) * self.scale
        ez = cols * U * (self.h.abs() @ self.w.abs().T)
        f = torch.finfo(TYPES[t])
        self.rel, self.sub = f.eps / 2, f.smallest_normal * f.eps / 2
        small = self.sub * 2.0 ** -13 * float(self.scale.max()) if t == "f16" else 0.0
        self.edz = (p * (torch.expm1(ez + 2 * U * x.abs()) + 4 * U) + 4 * U * self.hit) * self.scale \
            + self.rel ** 2 * self.dz.abs() * 1.01 + small * (self.scale > 0)

    def _grad(self, a, ea, b):
        want = a @ b
        e = ea @ b.abs() + (a.shape[1] + 256) * U * (a.abs() @ b.abs())
        return want, (e + self.rel * (want.abs() + e) + self.sub) * 1.001

    def off(self, dhidden, dweights):
        """How many elements of each gradient are outside the tolerance."""
        pairs = [(dhidden, self._grad(self.dz, self.edz, self.w)),
                 (dweights, self._grad(self.dz.T.contiguous(), self.edz.T.contiguous(), self.h))]
        return [int((~((got.double() - want).abs() <= tol)).sum()) for got, (want, tol) in pairs]
