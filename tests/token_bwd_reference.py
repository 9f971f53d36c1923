"""The token path's prologue gradients in fp64 torch, vectorised over tokens, for sizes that the oracle's loops over
tokens (oracle/token_path_backward.py) are too slow for; tests/test_token_bwd_reference.py holds the two together.

Beside the gradients it returns what an fp32 evaluation can be held to, row by row.  With c the relative accuracy of a
row of du (the convolution's gradient) against the row's scale G_t = r_t |dy_t| (r_t = 1 without the L2 norm; |.| the
norm over the row's channels, and |silu'| <= 1.1):

    |dx_t - exact| <= c sum_i max|tap_i| G_{t+i}

For |u| <= 16 at ordinary elements c = 1.2e-5 holds: the convolution's W + 1 <= 9 roundings of terms of size 16 move
silu' (|silu''| <= 0.5) by 9 * 2^-24 * 16 * 0.5 = 4.3e-6; the one-instruction exponential and reciprocal (2^-22 each)
with the argument's rounding (16 * 2^-24) and three roundings add 2e-6; the row sums (four terms in order, five
exchanges), the reciprocal root (2^-22) and four roundings 1.2e-6; the sum over the taps 1e-6; their first-order sum
is 8.5e-6.  Where |u| is far larger the sigmoid is 0 or 1 and silu' does not move at all.

A tap's gradients over a head's channels add up products of such a row and a row of x, so their error's norm is within
c sum_t G_t max|x_{t-i}|, and the additions themselves, of n terms in order, add n 2^-24 of the terms' absolute values,
which that sum bounds too.
"""
import torch

EPS = 1e-6
C = 1.2e-5


def places(cu, T, device):
    """Tokens since each token's sequence began, and tokens until it ends."""
    cu = torch.as_tensor(cu, dtype=torch.int64, device=device)
    t = torch.arange(T, device=device)
    seq = torch.searchsorted(cu, t, right=True) - 1
    return t - cu[seq], cu[seq + 1] - 1 - t


def _earlier(x, i, ok):
    y = torch.zeros_like(x)
    if i < x.shape[0]:
        y[i:] = x[:x.shape[0] - i]
    return torch.where(ok[:, None, None], y, 0.0)


def _later(x, i, ok):
    y = torch.zeros_like(x)
    if i < x.shape[0]:
        y[:x.shape[0] - i] = x[i:]
    return torch.where(ok.reshape(-1, *[1] * (x.dim() - 1)), y, torch.zeros((), dtype=x.dtype, device=x.device))


def prologue_gradients(x, taps, dy, cu, l2):
    """(dx [T, H, d], dtaps [H * d, W], the rows' bound / C [T, H], the tap gradients' bound / C [H, W]) of
    x [T, H, d], taps [H * d, W], dy [T, H, d]."""
    x, dy = x.double(), dy.double()
    T, H, d = x.shape
    wt = taps.double().reshape(H, d, -1)
    W = wt.shape[-1]
    age, left = places(cu, T, x.device)
    xs = [_earlier(x, i, age >= i) for i in range(W)]
    u = sum(wt[..., i] * xs[i] for i in range(W))
    sig = torch.sigmoid(u)
    ds, scale = dy, dy.norm(dim=-1)
    if l2:
        s = u * sig
        n = torch.sqrt((s * s).sum(-1, keepdim=True) + EPS)
        y = s / n
        ds = (dy - y * (y * dy).sum(-1, keepdim=True)) / n
        scale = scale / n[..., 0]
    du = ds * sig * (1 + u * (1 - sig))
    dx = sum(wt[..., i] * _later(du, i, left >= i) for i in range(W))
    bound = sum(wt[..., i].abs().amax(-1) * _later(scale, i, left >= i) for i in range(W))
    tap_bound = torch.stack([(scale * a.abs().amax(-1)).sum(0) for a in xs], -1)
    return dx, torch.stack([(du * a).sum(0) for a in xs], -1).reshape(H * d, W), bound, tap_bound
