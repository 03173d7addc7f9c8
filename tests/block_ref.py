"""Plain 64-bit forms of the operators around the long convolution, on the CPU;
gradients come from torch's autograd over them, not from the formulas."""
import torch


def half_step(dtype):
    """Largest relative error of one rounding to dtype."""
    return torch.finfo(dtype).eps / 2


def glr(v, f, g=None, bias=None, h0=None, reset=None, lens=None):
    """(y, h_last), position by position; y is 0 behind lens."""
    B, L, D = v.shape
    h = torch.zeros(B, D, dtype=torch.float64) if h0 is None else h0
    ys = []
    for t in range(L):
        a = torch.sigmoid(f[:, t] + (0 if bias is None else bias))
        prev = h
        if reset is not None:
            prev = torch.where(reset[:, t, None] != 0, torch.zeros_like(h), h)
        new = a * prev + torch.sigmoid(-(f[:, t] + (0 if bias is None else bias))) * v[:, t]
        y = new if g is None else new * g[:, t] * torch.sigmoid(g[:, t])
        if lens is not None:
            live = (t < lens)[:, None]
            new, y = torch.where(live, new, h), torch.where(live, y, torch.zeros_like(y))
        h = new
        ys.append(y)
    return torch.stack(ys, 1), h


def act(q, name):
    if name == "silu":
        return q * torch.sigmoid(q)
    if name == "gelu":
        return 0.5 * q * torch.special.erfc(-q / 2 ** 0.5)
    return q


def group_norm(x, G, gamma=None, beta=None, eps=1e-5, name="none", lens=None):
    """(y, mean, rstd) of x [B, S, C], sample by sample; y is 0 behind lens."""
    B, S, C = x.shape
    ys, means, rstds = [], [], []
    for b in range(B):
        n = S if lens is None else min(max(int(lens[b]), 0), S)
        xb = x[b, :n].reshape(n, G, C // G)
        mean = xb.mean((0, 2)) if n else x.new_zeros(G)
        var = (xb - mean[:, None]).square().mean((0, 2)) if n else x.new_zeros(G)
        rstd = 1 / torch.sqrt(var + eps)
        h = ((xb - mean[:, None]) * rstd[:, None]).reshape(n, C)
        h = h if gamma is None else h * gamma
        h = h if beta is None else h + beta
        ys.append(torch.cat([act(h, name), x.new_zeros(S - n, C)]))
        means.append(mean)
        rstds.append(rstd)
    return torch.stack(ys), torch.stack(means), torch.stack(rstds)


def ffn(x, w_in, w_out, name):
    """(y, z) of rows x [M, D]."""
    F = w_out.shape[0]
    pq = x @ w_in
    z = pq[:, :F] * act(pq[:, F:], name)
    return z @ w_out, z
