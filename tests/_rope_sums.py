"""Bounds for the weights' gradients of the norm and rotation that show a lost
row, a lost token and sums kept in 16 bits.

tests/_rope.py has what each row's term g' x r is off by.  The terms are added
in a tree whose depth is the number of additions that a term goes through, at
most: with G = 512 / d lane groups, 12 warps to each of 152 SMs and items of a
token or a share of its heads (there are at most tokens + 16 * 152 of them)
    a warp's items, for each the rows of a lane group and one more
                       ceil((tokens + 2432) / 1824) (ceil(heads / G) + 1)
    four warps of G lane groups                     4 G
    blocks, 32 lanes in turn, then the lanes        ceil(456 / 32) + 5.
Sums off by depth 2^-24 of the sum of magnitudes, where a bound for any order
has the number of rows."""
import torch

from _rope import T, backward_and_tol, turn

SMS = 152


def depth(tokens, heads, d):
    groups = 512 // d
    items = -(-(tokens + 16 * SMS) // (12 * SMS))
    return items * (-(-heads // groups) + 1) + 4 * groups + -(-3 * SMS // 32) + 5


def weight_grad_and_tol(dy, x, w, pos, inv_freq, eps, interleaved, amplitude):
    """(dw, tolerance, terms [B, heads, S, d]) of rows [B, heads, S, d]."""
    dx, dw, _, tol = backward_and_tol(dy, x, w, pos, inv_freq, eps, interleaved, amplitude)
    B, heads, S, d = x.shape
    terms = _terms(dy, x, pos, inv_freq, eps, interleaved, amplitude)
    assert torch.allclose(terms.sum((0, 1, 2)), dw, rtol=1e-9, atol=1e-9)
    size = terms.abs().sum((0, 1, 2))
    return dw, tol - B * heads * S * T * size + depth(B * S, heads, d) * T * size, terms


def _terms(dy, x, pos, inv_freq, eps, interleaved, amplitude):
    xd = x.double()
    r = 1.0 / torch.sqrt((xd * xd).mean(-1, keepdim=True) + eps)
    return turn(dy.double(), pos, inv_freq, interleaved, amplitude, back=True) * xd * r


# B, heads of q, of k, S, d, rot: short, long, several batch rows with several tokens to a warp
SHAPES = [(1, 1, 1, 2, 64, 16), (3, 7, 1, 5, 128, 48), (1, 28, 4, 333, 64, 16), (2, 3, 2, 700, 128, 112),
          (1, 8, 8, 2500, 64, 32), (1, 33, 31, 64, 128, 64), (3, 2, 1, 4001, 64, 64), (2, 1, 4, 3500, 128, 128),
          (5, 2, 2, 2047, 64, 48)]


def case(shape, dtype, seed=0):
    """CPU rows, gradients, weights, positions and frequencies."""
    B, H, H_kv, S, d, rot = shape
    g = torch.Generator().manual_seed(seed + S)
    x = {n: (torch.randn((B, h, S, d), generator=g) * scale).to(dtype)
         for n, h, scale in (("q", H, 1.5), ("k", H_kv, 0.7), ("dq", H, 1.0), ("dk", H_kv, 1.0))}
    x["pos"] = torch.randint(0, 5000, (B, S), generator=g).to(torch.int32)
    x["freq"] = (10000.0 ** (-torch.arange(rot // 2).double() * 2 / rot)).float()
    x["wq"], x["wk"] = torch.randn(d, generator=g), torch.randn(d, generator=g)
    return x
