"""Plain float64 forms of the gradient operators, and the error bounds that the
tests hold the kernels to.

Bounds.  A sum of c products in fp32 is off by at most c * u * sum |a||b|,
u = 2^-23 for each addition (half a step where the unit rounds, a whole one
where it cuts off); products of two bf16 are exact in fp32 and those of two
fp32 are inside the fused multiply-add.  The result is then rounded once to its
type: half a step, eps / 2 relative (bf16 2^-8, fp32 2^-24).
"""

import numpy as np
import torch

U = 2.0 ** -23


def half_step(dtype):
    return torch.finfo(dtype).eps / 2


def f64(t):
    return t.detach().to("cpu", torch.float64)


def segments(offsets, rows):
    off = [int(v) for v in offsets]
    return [(off[e], off[e + 1]) for e in range(len(off) - 1)]


def linear(x, w, offsets):
    """(value, sum of magnitudes, covered rows) of the forward product."""
    x, w = f64(x), f64(w)
    y = torch.zeros(x.shape[0], w.shape[1], dtype=torch.float64)
    mag, on = torch.zeros_like(y), torch.zeros(x.shape[0], dtype=torch.bool)
    for e, (lo, hi) in enumerate(segments(offsets, x.shape[0])):
        y[lo:hi] = x[lo:hi] @ w[e].t()
        mag[lo:hi] = x[lo:hi].abs() @ w[e].abs().t()
        on[lo:hi] = True
    return y, mag, on


def dgrad(dy, w, offsets):
    return linear(dy, f64(w).transpose(1, 2).contiguous(), offsets)


def wgrad(dy, x, offsets):
    dy, x = f64(dy), f64(x)
    segs = segments(offsets, dy.shape[0])
    dw = torch.stack([dy[lo:hi].t() @ x[lo:hi] for lo, hi in segs])
    mag = torch.stack([dy[lo:hi].abs().t() @ x[lo:hi].abs() for lo, hi in segs])
    terms = torch.tensor([hi - lo for lo, hi in segs], dtype=torch.float64)
    return dw, mag, terms


def worst(got, want, bound):
    """Largest |got - want| / bound (0 where both are equal)."""
    d = (f64(got) - want).abs()
    r = torch.where(d == 0, torch.zeros_like(d), d / bound)
    assert not torch.isnan(d).any(), "NaN in the result"
    return float(r.max()) if r.numel() else 0.0


def ckpt_quantize(x):
    """(codes, scales) as numpy, by the rule: 2^e the smallest power of two,
    e >= -126, with max |x| <= 127 * 2^e, and 121 at most; ties to even."""
    x = f64(x).numpy()
    rows, k = x.shape
    nb = -(-k // 128)
    codes, scales = np.zeros((rows, k), np.int8), np.zeros((rows, nb), np.uint8)
    for b in range(nb):
        v = x[:, b * 128:(b + 1) * 128]
        bad = ~np.isfinite(v).all(1)
        top = np.where(bad, 0.0, np.abs(np.where(np.isfinite(v), v, 0.0)).max(1))
        m, p = np.frexp(top)
        e = np.clip(np.where(top == 0, -126, p - 7 + (m > 127.0 / 128.0)), -126, 121)
        q = np.clip(np.rint(np.where(bad[:, None], 0.0, v) * np.ldexp(1.0, -e)[:, None]), -127, 127)
        codes[:, b * 128:(b + 1) * 128] = q
        scales[:, b] = np.where(bad, 255, e + 127)
    return codes, scales


def ckpt_restore(codes, scales):
    k = codes.shape[1]
    s = np.where(scales == 255, np.nan, np.ldexp(1.0, scales.astype(np.int64) - 127))
    return codes.astype(np.float64) * np.repeat(s, 128, axis=1)[:, :k]


def embedding(table, tokens, scale):
    t = tokens.cpu().reshape(-1).long()
    on = (t >= 0) & (t < table.shape[0])
    out = torch.zeros(t.numel(), table.shape[1], dtype=torch.float64)
    out[on] = f64(table)[t[on]] * float(np.float32(scale))
    return out


def embedding_grad(dy, tokens, vocab, scale):
    """(sum * scale, sum of magnitudes * |scale|, number of terms per row)"""
    t = tokens.cpu().reshape(-1).long()
    on = (t >= 0) & (t < vocab)
    s = float(np.float32(scale))
    g = torch.zeros(vocab, dy.shape[1], dtype=torch.float64)
    mag = torch.zeros_like(g)
    g.index_add_(0, t[on], f64(dy)[on] * s)
    mag.index_add_(0, t[on], (f64(dy)[on] * s).abs())
    return g, mag, torch.bincount(t[on], minlength=vocab).double()
