"""64-bit references of the few-token operators, each with an elementwise bound
on a correct kernel's error (test infrastructure).

Bounds.  u = 2^-23 bounds the error of one float32 addition or product (half a
step is 2^-24; the matrix cores may truncate), so a float32 sum of n products
is within n u sum|a b| of the exact one.  A bf16 rounding is within 2^-8 of the
value; a hidden value kept as a bf16 number and its bf16 remainder within
2^-16.  |GELU'| and |SiLU'| stay below 1.13.  The activation itself and the
routing weight (an exponential, a quotient, a product; the logits' difference
rounded to float32) add at most 2^-18 of the value.

4-bit groups of up to 128 form sum (128 + q) x - sum 136 x + (8 - z) sum x in
float32 before the scale: 256 products with factors up to 143, and the last
term at most 8 / 136 of the second, within 256 u 300 sum|x|.
"""
import torch

U = 2.0 ** -23
F64 = torch.float64


def unpack_w4(codes, scales, zeros):
    """(values, per-k scale) in 64 bits."""
    q = torch.stack((codes & 15, codes >> 4), dim=-1).flatten(-2).to(F64)
    rep = q.shape[-1] // scales.shape[-1]
    s = scales.to(F64).repeat_interleave(rep, -1)
    z = 8.0 if zeros is None else (zeros & 15).to(F64).repeat_interleave(rep, -1)
    return s * (q - z), s


def dot_bound(a, w, w_scale=None):
    """Bound of float32 sums a [M, K] w [N, K]^T (4-bit: w_scale [N, K])."""
    n = a.shape[1] + 16
    b = n * U * (a.abs() @ w.abs().t())
    if w_scale is not None:
        b = b + 256 * U * 300 * (a.abs() @ w_scale.abs().t())
    return b


def act(v, name):
    if name == "silu":
        return v * torch.sigmoid(v)
    return v * 0.5 * torch.erfc(-v / 2.0 ** 0.5)


def layer(x, W_g, expert, E, k, S, b_g, b_sel, activation, out_half_step, hidden_bits):
    """Everything on the CPU.  expert(e) -> (W1, scale1 or None, b1 or None, W2, scale2 or None, b2 or None) in 64 bits.
    Returns out, idx, w, bound."""
    x = x.to(F64)
    T, d = x.shape
    logits = x @ W_g.to(F64).t()
    if b_g is not None:
        logits = logits + b_g.to(F64)
    key = logits if b_sel is None else logits + b_sel.to(F64)
    key = torch.where(key.isnan(), torch.full_like(key, -torch.inf), key)
    idx = torch.sort(key, dim=1, descending=True, stable=True).indices[:, :k]
    w = torch.softmax(torch.gather(logits, 1, idx), dim=1)
    out = torch.zeros(T, d, dtype=F64)
    bound = torch.zeros(T, d, dtype=F64)
    for e in range(E + S):
        if e < E:
            hit = (idx == e)
            tok = hit.any(1).nonzero().flatten()
            g = (w * hit).sum(1)[tok]
        else:
            tok, g = torch.arange(T), torch.ones(T, dtype=F64)
        if tok.numel() == 0:
            continue
        W1, s1, b1, W2, s2, b2 = expert(e)
        u = x[tok] @ W1.t()
        eu = dot_bound(x[tok], W1, s1)
        if b1 is not None:
            u = u + b1
            eu = eu + U * (u.abs() + b1.abs())
        a = act(u, activation)
        ea = 1.13 * eu + (hidden_bits + 2.0 ** -18) * a.abs()
        y = a @ W2.t()
        ey = ea @ W2.abs().t() + dot_bound(a.abs() + ea, W2, s2) + (k + S) * U * y.abs()
        if b2 is not None:
            y = y + b2
            ey = ey + (k + S + 2) * U * b2.abs() + 2.0 ** -18 * b2.abs()
        out.index_add_(0, tok, g[:, None] * y)
        bound.index_add_(0, tok, g[:, None] * ey)
    # the shares of a column are added in float32 too
    bound = bound * (1 + 64 * U) + 64 * U * out.abs()
    return out, idx, w, bound + out_half_step * (out.abs() + bound)


def check(got, want, bound, what):
    got = got.to(F64).cpu()
    assert torch.isfinite(got).all(), what
    over = (got - want).abs() - bound - 1e-30
    worst = int(over.argmax())
    assert over.max() <= 0, (what, worst, float(got.flatten()[worst]), float(want.flatten()[worst]),
                             float(bound.flatten()[worst]))
