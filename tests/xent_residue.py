"""A cross entropy call whose gradients are those of the targets' logits: what 16 bits lose of a
target's dz shows in them, unless it is given back.

Tolerances, with u = 2^-24 and r, s the relative and absolute half steps of the type:
- dz of a target is (p - 1) dloss in f32: off by what the logit's error makes of p, and 4 u.
  Nothing is added for a rounding to 16 bits: what that takes has to be given back;
- dz of another row is rounded once: r of itself (f16: and s of the largest dloss / 2^14);
- a gradient is off by its terms' errors, by (n + 256) u of its n terms' sizes, and by r and s
  for its rounding.
"""
import torch

TYPES = {"f16": torch.float16, "bf16": torch.bfloat16}
U = 2.0 ** -24


class Targets:
    """Hidden states are zero in the second half of the columns, and there only the targets'
    rows have weights, so that a token's gradient there is its target's dz times a weight and
    little else; a target's row of the weight gradient sums its own tokens."""

    def __init__(self, tokens, rows, cols, t, seed, device):
        g = torch.Generator(device=device)
        g.manual_seed(seed)
        n = lambda *s: torch.randn(*s, generator=g, device=device)  # noqa: E731
        self.tokens, self.rows, self.cols, self.t = tokens, rows, cols, t
        vocab, half = sum(rows), cols // 2
        # rows of both halves of a 256-row tile, its ends, and the last shard's last
        self.wanted = torch.tensor(sorted({3, 126, 127, 128, 200, 255, rows[0] - 1, vocab - 1}), device=device)
        hidden, weights = n(tokens, cols), n(vocab, cols) / cols ** 0.5
        hidden[:, half:] = 0.0
        weights[:, half:] = 0.0
        weights[self.wanted, half:] = n(len(self.wanted), half)
        self.hidden, weights = hidden.to(TYPES[t]), weights.to(TYPES[t])
        self.weights = [w.contiguous() for w in weights.split(rows)]
        self.targets = self.wanted[torch.randint(0, len(self.wanted), (tokens,), generator=g, device=device)]
        self.dloss = 0.5 + torch.rand(tokens, generator=g, device=device)
        self.h, self.w = self.hidden.double(), torch.cat(self.weights).double()
        z = self.h @ self.w.T
        self.lse = torch.logsumexp(z, 1).float()
        x = z - self.lse.double()[:, None]
        p = x.exp()
        dl = self.dloss.double()[:, None]
        self.hit = torch.zeros_like(p).scatter_(1, self.targets[:, None], 1.0)
        self.dz = (p - self.hit) * dl
        ez = cols * U * (self.h.abs() @ self.w.abs().T)
        f = torch.finfo(TYPES[t])
        self.rel, self.sub = f.eps / 2, f.smallest_normal * f.eps / 2
        step = self.rel * self.dz.abs() * 1.01
        if t == "f16":
            step = step + self.sub * 2.0 ** -13 * float(dl.max())
        self.edz = (p * (torch.expm1(ez + 2 * U * x.abs()) + 4 * U) + 4 * U * self.hit) * dl + torch.where(self.hit > 0, 0.0, step)

    def _grad(self, a, ea, b):
        want = a @ b
        e = ea @ b.abs() + (a.shape[1] + 256) * U * (a.abs() @ b.abs())
        return want, (e + self.rel * (want.abs() + e) + self.sub) * 1.001

    def expected(self):
        """(value, tolerance) of dhidden, and of all shards' dweights together."""
        return self._grad(self.dz, self.edz, self.w), self._grad(self.dz.T.contiguous(), self.edz.T.contiguous(), self.h)

    def share_off(self, dhidden, dweights):
        """Shares of the targets' part of dhidden and dweights that are outside the tolerance."""
        (dh, eh), (dw, ew) = self.expected()
        half = self.cols // 2
        off = [~((dhidden.double() - dh).abs() <= eh)[:, half:], ~((dweights.double() - dw).abs() <= ew)[self.wanted, :half]]
        return [float(x.double().mean()) for x in off]
