"""Inputs and 64-bit definitions for the tests of the microscaled 4-bit
operators (E2M1 codes in blocks of 32 along a row, one E8M0 scale each)."""
import torch

from expert_util import H, TINY

MAGNITUDES = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)


def bytes_like(t, extra=0):
    """t (uint8) in storage whose row pitch is a multiple of 16 bytes, the
    padding filled with 0xff: scales there would be NaN, codes -6."""
    ld = (-(-t.shape[-1] // 16) + extra) * 16
    big = torch.full(t.shape[:-1] + (ld,), 255, dtype=torch.uint8, device="cuda")
    out = big[..., :t.shape[-1]]
    out.copy_(t)
    return out


def random_blocks(shape, seed, lo=120, hi=130, extra=0):
    """Random codes and scales (exponents lo..hi) of shape[:-1] rows of K values."""
    g = torch.Generator().manual_seed(seed)
    K = shape[-1]
    q = torch.randint(0, 256, shape[:-1] + (-(-K // 2),), generator=g, dtype=torch.uint8)
    if K % 2:
        q[..., -1] &= 15
    s = torch.randint(lo, hi + 1, shape[:-1] + (-(-K // 32),), generator=g, dtype=torch.uint8)
    return bytes_like(q, extra), bytes_like(s, extra)


def values(q, s, K=None):
    """The values of codes and scales in 64 bits; NaN for scale 255."""
    table = torch.tensor(MAGNITUDES + tuple(-v for v in MAGNITUDES), dtype=torch.float64, device=q.device)
    v = torch.stack((table[(q & 15).long()], table[(q >> 4).long()]), -1).flatten(-2)
    up = ((s.long() + (1023 - 127)) << 52).view(torch.float64)
    up = torch.where(s == 255, torch.nan, up)
    v = v * up.repeat_interleave(32, -1)[..., :v.shape[-1]]
    return v if K is None else v[..., :K]


def quantised(X):
    """(codes, scales) of the rows of X, by the definition, as Python sees it:
    on the host in 64 bits, the nearest magnitude, ties to the even code."""
    X = X.detach().cpu().double()
    M, K = X.shape
    nb = -(-K // 32)
    b = torch.nn.functional.pad(X, (0, nb * 32 - K)).view(M, nb, 32)
    top = b.abs().amax(2)
    bad = ~torch.isfinite(b).all(2)
    _, e = torch.frexp(torch.where(bad, 1.0, top))
    E = torch.where(top > 0, (e - 3 + 127).clamp(min=0), 0)
    y = torch.where(bad[..., None], 0.0, b) / ((E.long() + (1023 - 127)) << 52).view(torch.float64)[..., None]
    mags = torch.tensor(MAGNITUDES, dtype=torch.float64)
    d = (y.abs()[..., None] - mags).abs()
    near = d.amin(-1, keepdim=True)
    hit = d == near                                    # one code, or two neighbours of a tie
    lower = hit.long().argmax(-1)
    code = torch.where((hit.sum(-1) == 2) & (lower % 2 == 1), lower + 1, lower)
    code = torch.where(torch.signbit(y), code + 8, code)
    code = torch.where(bad[..., None], 0, code).view(M, nb * 32)[:, :K]
    code = torch.nn.functional.pad(code, (0, K % 2)).view(M, -1, 2)
    return ((code[..., 0] | code[..., 1] << 4).to(torch.uint8),
            torch.where(bad, 255, E).to(torch.uint8))


def product(a, w, dtype):
    """a @ w.T in 64 bits (a, w values), and the bound of an fp32 sum of exact
    products in any order, rounded once to dtype."""
    ref = a @ w.t()
    return ref, H[dtype] * ref.abs() * 1.01 + TINY[dtype] + a.shape[1] * 2.0 ** -23 * (a.abs() @ w.abs().t())
