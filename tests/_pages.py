"""Plain 64-bit forms of the page operators, for the tests (torch, any device).

A cache is a dict: ``rows`` [n_rows][576] float64 values as the pool stands for
them, ``table`` int [R][P] GPU blocks (-1: none), ``ctx`` list of lengths."""
import math

import torch

PAGE, DIM, NOPE = 64, 576, 512


def quantise(x):
    """BF16 rows (any shape [..., 576]) to e4m3 codes and scales as the pool defines them."""
    f = x.float()
    amax = f.abs().amax(-1)
    scale = amax / torch.full_like(amax, 448.0)
    scale = torch.maximum(scale, torch.full_like(scale, 2.0 ** -126))
    bad = ~torch.isfinite(f).all(-1)
    scale = torch.where(bad, torch.full_like(scale, math.nan), scale)
    # quotients in 64 bits, rounded to 32 as the definition has it
    q = (f.double() / scale[..., None].double()).float()
    return q.to(torch.float8_e4m3fn), scale


def values(codes_u8, scales=None):
    """Pool rows (uint8 [n][row_bytes]) as float64 values."""
    if scales is None:
        return codes_u8.view(torch.bfloat16).double()
    return codes_u8.view(torch.float8_e4m3fn).float().double() * scales.double()[:, None]


def seen_mask(L, T, tree, t):
    """Bool [L]: the positions that query token t sees."""
    pos = torch.arange(L)
    if tree is None:
        return pos <= L - T + t
    node = pos - (L - T)
    m = int(tree[t]) & ((1 << 64) - 1)
    bits = torch.tensor([bool(m >> i & 1) for i in range(T)] + [False])
    return (node < 0) | bits[node.clamp(-1, T - 1)] & (node >= 0)


def attention(q, kv, keep, scale):
    """q [H][576], kv [K][576], keep [K] bool, all float64. Returns out [H][512], lse [H],
    mass [H][512] (the weighted mean of |value|: what a relative error of the weights
    can move) and reach (a bound on |scale q.k|)."""
    if not bool(keep.any()):
        H = q.shape[0]
        z = torch.zeros(H, NOPE, dtype=torch.float64, device=q.device)
        return z, torch.full((H,), -math.inf, dtype=torch.float64, device=q.device), z.clone(), 0.0
    k = kv[keep]
    x = q @ k.T * scale
    w = torch.softmax(x, -1)
    reach = abs(scale) * float(q.norm(dim=1).max() * k.norm(dim=1).max())
    return w @ k[:, :NOPE], torch.logsumexp(x, -1), w @ k[:, :NOPE].abs(), reach


def check_attention(out, lse, ref, ref_lse, mass, reach, what=""):
    """out and lse of one query token's heads against the 64-bit form.

    Roundings, each at most half a step: the output to BF16 (2^-8 of it), each
    weight to BF16 (2^-8 of the weighted mean of |value|). Scores are 32-bit sums:
    their error is taken as 2^-16 of |q||k| (36 MMAs that each cut 16 products and the
    sum so far at 2^-25 of the largest's power of two lose 2^-16 of a product that is
    all of |q||k|; products of like size are far smaller), which moves a weight by that
    and the sum of the weights by as much again; exp, the split's join and the division
    stay below 2^-18."""
    e = reach * 2.0 ** -16 + 2.0 ** -18
    tol = 2.0 ** -8 * (ref.abs() + mass) * (1 + 2.0 ** -7) + 2 * e * mass + 1e-30
    d = (out.double() - ref).abs()
    assert torch.isfinite(out).all(), what
    assert bool((d <= tol).all()), f"{what}: out off by {float((d / tol).max()):.3f} of the tolerance"
    fin = torch.isfinite(ref_lse)
    assert bool((torch.isfinite(lse) == fin).all()), what
    dl = (lse.double() - ref_lse)[fin].abs()
    tl = e + 2.0 ** -20 * (1 + ref_lse[fin].abs())
    assert bool((dl <= tl).all()), f"{what}: lse off by {float((dl / tl).max()):.3f} of the tolerance"


def select(q, means, n_candidates, N, n_first, n_last):
    """q [H][576], means [P][576] float64: the chosen pages, ascending, as a list."""
    if n_candidates <= N:
        return list(range(n_candidates))
    s = (q @ means[:n_candidates].T)
    s = torch.where(torch.isnan(s), torch.full_like(s, -math.inf), s).amax(0)
    forced = set(range(n_first)) | set(range(n_candidates - n_last, n_candidates))
    rest = [p for p in torch.argsort(s, descending=True, stable=True).tolist() if p not in forced]
    return sorted(forced | set(rest[:N - len(forced)]))
