"""64-bit reference of the packed attention calls and of rotary positions, with
the error bounds that the kernels' arithmetic implies."""
import math

import torch

HALF_STEP = {torch.bfloat16: 2.0 ** -8, torch.float32: 2.0 ** -24}


class Ref:
    """O, lse in 64 bits and elementwise bounds on |kernel - reference|.

    Per row: s_j the logits, p_j = e^(s_j - lse), A = sum_j p_j |v_j|.
      logits   fp32 sums of d products, each addition off by at most 2^-23 of the
               running magnitude (tensor cores may truncate): |ds| <= (d + 8) 2^-23
               scale sum_c |q_c k_c| =: e, the + 8 covers scaling and the subtraction
      p        relative e^(2 e) - 1 + 2^-20 (approximate exponential); in bf16
               kernels also 2^-8, p's rounding
      sums     n 2^-23 relative to A and to the normaliser
      O        half a step of the output type relative to O
      lse      e + 2^-20 + n 2^-23, and 2^-22 |lse| for its last operations
    """

    def __init__(self, Q, K, V, q_lens, kv_lens, kv_starts=None, causal=True, Kp=None, Vp=None,
                 scale=None):
        t, h, d = Q.shape
        hk = K.shape[1] if K is not None else Kp.shape[1]
        g = h // hk
        pre = 0 if Kp is None else Kp.shape[0]
        scale = 1 / math.sqrt(d) if scale is None else scale
        rows = sum(q_lens)
        dev = Q.device
        self.O = torch.zeros(rows, h, d, dtype=torch.float64, device=dev)
        self.lse = torch.full((rows, h), -torch.inf, dtype=torch.float64, device=dev)
        self.O_tol, self.lse_tol = torch.zeros_like(self.O), torch.zeros_like(self.lse)
        half = HALF_STEP[Q.dtype]
        p_round = half if Q.dtype == torch.bfloat16 else 0.0
        at = end = 0
        for s, (n, m) in enumerate(zip(q_lens, kv_lens)):
            k0 = end if kv_starts is None else kv_starts[s]
            end += m
            if n == 0:
                continue
            ks, vs = [], []
            if pre:
                ks.append(Kp)
                vs.append(Vp)
            if m:
                ks.append(K[k0:k0 + m])
                vs.append(V[k0:k0 + m])
            if not ks:
                at += n
                continue
            k, v = torch.cat(ks).double(), torch.cat(vs).double()
            j = torch.arange(pre + m, device=dev) - pre
            i = torch.arange(n, device=dev)
            seen = (j[None] < 0) | (j[None] <= i[:, None] + m - n) if causal else \
                torch.ones(n, pre + m, dtype=torch.bool, device=dev)
            q = Q[at:at + n].double()
            for head in range(h):
                kh, vh, qh = k[:, head // g], v[:, head // g], q[:, head]
                S = torch.where(seen, scale * (qh @ kh.T), -torch.inf)
                e = torch.where(seen, abs(scale) * (qh.abs() @ kh.abs().T), 0.0).amax(-1)
                e = e * (d + 8) * 2.0 ** -23
                lse = torch.logsumexp(S, -1)
                P = torch.exp(S - torch.where(torch.isinf(lse), 0.0, lse)[:, None])
                P = torch.where(seen, P, 0.0)
                # masked keys drop out whatever they hold
                vz = torch.where(seen.any(0)[:, None], vh, 0.0)
                bad = ~torch.isfinite(vz).all(-1)
                O = P[:, ~bad] @ vz[~bad]
                A = P[:, ~bad] @ vz[~bad].abs()
                for b in bad.nonzero().flatten().tolist():  # non-finite values where seen
                    add = torch.where(torch.isfinite(vz[b]), P[:, b:b + 1] * vz[b], vz[b])
                    O = O + torch.where(seen[:, b:b + 1], add, 0.0)
                    A = A + torch.where(seen[:, b:b + 1], vz[b].abs(), 0.0)
                count = (pre + m) * 2.0 ** -23
                rel = torch.expm1(2 * e) + 2.0 ** -20 + p_round + 2 * count
                self.O[at:at + n, head] = O
                self.lse[at:at + n, head] = lse
                self.O_tol[at:at + n, head] = half * O.abs() + (1 + half) * rel[:, None] * A
                self.lse_tol[at:at + n, head] = torch.where(
                    torch.isinf(lse), 0.0, e + 2.0 ** -20 + count + 2.0 ** -22 * lse.abs())
            at += n

    def check(self, O, lse=None):
        rows = self.O.shape[0]
        self._same(O[:rows].double(), self.O, self.O_tol, "O")
        if lse is not None:
            self._same(lse[:rows].double(), self.lse, self.lse_tol, "lse")

    @staticmethod
    def _same(x, ref, tol, what):
        fine = torch.isfinite(ref)
        assert torch.equal(torch.isnan(x), torch.isnan(ref)), f"{what}: NaN where there is none"
        inf = torch.isinf(ref)
        assert torch.equal(x[inf], ref[inf]), f"{what}: infinities differ"
        off = (x - ref).abs()[fine]
        over = off > tol[fine]
        assert not over.any(), (f"{what}: {int(over.sum())} of {over.numel()} values out of bounds, "
                                f"worst {float((off - tol[fine]).max()):.3g} over, "
                                f"largest difference {float(off.max()):.3g}")


def rotary_tables(head_dim, rotary_dim, positions, base=10000.0, scaling=None, factor=1.0,
                  original_len=0.0, fast=32.0, slow=1.0, sections=None):
    """cos and sin (64 bits) [tokens..., pairs] and the amplitude, from the formulas.
    positions: [axes, ...] integers."""
    pairs = rotary_dim // 2
    sections = [pairs] if sections is None else sections
    cols = []
    for a, s in enumerate(sections):
        for i in range(s):
            b = base * factor ** (s / (s - 1)) if scaling == "base" and s > 1 else base
            w = b ** (-i / s)
            if scaling == "linear":
                w /= factor
            if scaling == "ramp":
                c = min(1.0, max(0.0, (original_len * w / (2 * math.pi) - slow) / (fast - slow)))
                w = c * w + (1 - c) * w / factor
            cols.append(positions[a].double() * w)
    ang = torch.stack(cols, -1)
    return ang.cos(), ang.sin(), 1 + 0.1 * math.log(factor) if scaling == "ramp" else 1.0


def rotary_ref(x, cos, sin, amp, rotary_dim, layout, backward=False):
    """y in 64 bits and the bound on a kernel's error: cos and sin off by at most 2^-21 (the
    angle in half turns rounded to 24 bits, pi 2^-24, and the functions' own two units), three
    fp32 roundings, and half a step of the output type."""
    half = rotary_dim // 2
    first = slice(0, half) if layout == "half" else slice(0, rotary_dim, 2)
    second = slice(half, rotary_dim) if layout == "half" else slice(1, rotary_dim, 2)
    f = x.double()
    y = f.clone()
    s = -sin if backward else sin
    a, b = f[..., first], f[..., second]
    y[..., first] = amp * (a * cos - b * s)
    y[..., second] = amp * (b * cos + a * s)
    tol = torch.zeros_like(y)
    tol[..., first] = tol[..., second] = amp * (a.abs() + b.abs()) * (2.0 ** -21 + 3 * 2.0 ** -24)
    return y, tol + HALF_STEP[x.dtype] * y.abs() * (torch.arange(x.shape[-1], device=x.device)
                                                    < rotary_dim)
