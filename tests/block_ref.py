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
