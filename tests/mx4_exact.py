"""MXFP4 inputs whose products have exact sums, and their 64-bit results in
torch on whatever device the inputs are (the numpy forms of mx_ref.py are too
slow for a kernel's largest tiles; test_mx4_launches.py holds these to them).

Every code is a multiple of 1/2, so with scale bytes of at least lo_w and lo_x
every product, and every partial sum in any order, is a multiple of
2^(lo_w + lo_x - 254) / 4.  No partial sum passes A = sum |w x|.  Where 4 A /
2^(lo_w + lo_x - 254) is below 2^24, fp32 holds all of them: the result is the
same bit for bit whatever the order, and one lost, doubled or misplaced block
shows.  ``held`` checks that bound for the inputs at hand.
"""
import torch

E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0, -0.0, -0.5, -1.0, -1.5, -2.0, -3.0, -4.0, -6.0)
W_LO, X_LO = 120, 130                                          # scale bytes lo .. lo + 2


def codes(g, lead, K, lo, spread=3):
    """(codes, scale bytes) of rows of K values, random."""
    kw = dict(dtype=torch.uint8, device=g.device, generator=g)
    return (torch.randint(0, 256, lead + (K // 2,), **kw), torch.randint(lo, lo + spread, lead + (K // 32,), **kw))


def values(c, s):
    """The values [..][K] in 64 bits; scale byte 255 is NaN."""
    lut = torch.tensor(E2M1, dtype=torch.float64, device=c.device)
    pair = torch.stack((lut.repeat(16), lut.repeat_interleave(16)), dim=1)     # of a code byte: low, high nibble
    v = pair[c.int()].reshape(s.shape + (32,))
    p = ((s.long() + (1023 - 127)) << 52).view(torch.float64)
    p = torch.where(s == 255, torch.full_like(p, float("nan")), p)
    return (v * p[..., None]).flatten(-2)


def held(A, w_lo=W_LO, x_lo=X_LO, parts=4):
    """Every partial sum is a whole number of 1/parts of the smallest step, below 2^24 of them."""
    most = A.max().item()
    assert most * parts / 2.0 ** (w_lo + x_lo - 254) < 2.0 ** 24, most


def dense(c, s, x):
    """(y, A): x (M, K) times the rows (c, s) (N, K), and the sums of the magnitudes.  A few rows at a time: of more
    than 2^26 pairs of the look-up in ``values`` torch wrote the first n % 2^26 only (measured: 8300 x 8192 codes)."""
    y = torch.empty(x.shape[0], c.shape[0], dtype=torch.float64, device=c.device)
    A = torch.empty_like(y)
    some = max(1, (1 << 25) // x.shape[1])
    for n in range(0, c.shape[0], some):
        w = values(c[n:n + some], s[n:n + some])
        y[:, n:n + some], A[:, n:n + some] = x @ w.t(), x.abs() @ w.abs().t()
    return y, A


def gather(ids, c, s, x):
    """(y, A) (M, top_k, N) of x (M, K) or (M, top_k, K); zeros where an id is outside [0, E)."""
    y = torch.zeros(*ids.shape, c.shape[1], dtype=torch.float64, device=c.device)
    A = torch.zeros_like(y)
    for e in range(c.shape[0]):
        t, j = torch.nonzero(ids == e, as_tuple=True)
        if t.numel():
            y[t, j], A[t, j] = dense(c[e], s[e], x[t, j] if x.dim() == 3 else x[t])
    return y, A


def make_ids(g, M, top_k, E, holes=True, skew=False):
    """Expert ids, an eighth of them outside [0, E); skewed: half of the pairs go to two experts."""
    ids = torch.randint(0, E, (M, top_k), device=g.device, generator=g)
    p = torch.rand(M, top_k, device=g.device, generator=g)
    if skew:
        ids = torch.where(p < 0.5, ids % 2, ids)
    if holes:
        out = torch.tensor([-1, E, 2 ** 31 - 1, -2 ** 31], device=g.device)
        ids = torch.where(p > 0.875, out[ids % 4], ids)
    return ids.int()
