"""The selective state-space mixer's operators in plain float64 (CPU torch),
written from their definitions, with a bound on the magnitudes that enter each
sum, from which the tests derive how far fp32 arithmetic may be off.

Rounding model. Per token a state is multiplied by one decay and gets one
product added: the decay's exponential is off by at most 2^-22.5 and its
argument by 2^-23 |argument| with |argument| <= 8 where the decay still
matters (below e^-8 the product's weight is itself below 4e-4 of that bound),
the multiply-adds by 2^-24 each. That is under STEP = 2e-6 relative a token, a
contribution that is k tokens old carries at most k of them, and every sum of
terms t_i is off by at most STEP * tokens * sum |t_i|. The bounds are taken
relative to sums of absolute values ("mag"), so cancellation is covered."""
import torch

STEP = 2e-6
F64 = torch.float64


def half_step(dtype):
    return torch.finfo(dtype).eps / 2


def d(t):
    return None if t is None else t.detach().cpu().to(F64)


def softplus(v):
    return torch.logaddexp(v, torch.zeros_like(v))


def silu(v):
    return v * torch.sigmoid(v)


def conv(x, w, b, win):
    """x [T, D], win [4, D] (oldest first): u, the sum of magnitudes, the new window."""
    rows = torch.cat([win, x])
    T = x.shape[0]
    acc = sum(rows[1 + j:1 + j + T] * w[:, j] for j in range(4)) + (0 if b is None else b)
    mag = sum((rows[1 + j:1 + j + T] * w[:, j]).abs() for j in range(4)) + (0 if b is None else b.abs())
    return silu(acc), 1.1 * mag, rows[-4:]


def scan(x, dt, A, Bm, Cm, skip, z, bias, h, soft=True, umag=None):
    """One sequence: x [T, D] (u), h [D, N]. Returns y, its magnitudes, the
    last state and its magnitudes. The operands must be float64."""
    T = x.shape[0]
    delta = dt + (0 if bias is None else bias)
    if soft:
        delta = softplus(delta)
    umag = x.abs() if umag is None else umag
    hm = h.abs()
    y, ym = torch.empty_like(x), torch.empty_like(x)
    for t in range(T):
        a = torch.exp(delta[t][:, None] * A)
        h = a * h + (delta[t] * x[t])[:, None] * Bm[t]
        hm = a * hm + (delta[t].abs() * umag[t])[:, None] * Bm[t].abs()
        y[t] = (h * Cm[t]).sum(-1)
        ym[t] = (hm * Cm[t].abs()).sum(-1)
    if skip is not None:
        y = y + skip * x
        ym = ym + skip.abs() * umag
    if z is not None:
        g = silu(z)
        y, ym = y * g, ym * g.abs()
    return y, ym, h, hm


def close(got, ref, mag, tokens, name=""):
    """got (device tensor, its type's rounding) against ref (float64) within the model above."""
    g = d(got)
    assert g.shape == ref.shape, (name, g.shape, ref.shape)
    assert torch.equal(torch.isnan(g), torch.isnan(ref)), f"{name}: NaN in other places"
    ok = ~torch.isnan(ref)
    tol = half_step(got.dtype) * ref.abs() + STEP * (tokens + 8) * mag + 1e-30
    over = ((g - ref).abs() - tol)[ok]
    assert over.numel() == 0 or over.max() <= 0, f"{name}: off by up to {float(((g - ref).abs() / tol)[ok].max()):.3g} of the bound"
