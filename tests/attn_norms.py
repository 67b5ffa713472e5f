"""Checks of attention that see a lost block of keys or a part of wrong weight, however many keys there are."""
import torch

# Of a token's head: the result is rounded to bf16 (at most 2^-8 of each element, so of the norm).  Each
# probability is rounded to bf16 for its product with v, at most 2^-8 of it; over values of no mean, independent
# of the roundings, that moves the output by 2^-8 sqrt(sum p^2 |v|^2) at most, and the output's own norm is
# sqrt(sum p^2 |v|^2) give or take a factor of two in the smallest of thousands of heads of 64 or more elements.
NORM = 2.0 ** -8 + 2 * 2.0 ** -8


def norm_errors(got, ref):
    """Relative error of every (token, head): [T][hq]; heads of no keys must be zeros."""
    size = ref.norm(dim=-1)
    diff = (got - ref).norm(dim=-1)
    return torch.where(size == 0, torch.where(diff == 0, 0.0, float("inf")), diff / size)


def check_norms(b, ref=None):
    """`b` has run: every token's head within NORM of the 64-bit one, and within b.check()'s bounds."""
    ref = ref if ref is not None else b.reference()
    b.check(ref)
    got = b.out[:b.T, :b.hq * b.d].double().cpu().view(b.T, b.hq, b.d)
    e = norm_errors(got, ref[0])
    assert torch.all(e <= NORM), f"{float(e.max()):.3e} at {(e == e.max()).nonzero()[0].tolist()}"


def single_out(b, block=128):
    """Values of zero but for the keys on both sides of every block's boundary and the first and last ones, which
    have a one each, on elements that follow each other: a lost or misplaced key changes an element by its whole
    weight, and b.check()'s bounds, with no cancellation in them, are 2^-7 of each element."""
    for line, rows in enumerate(b.place):
        n = len(rows)
        b.v[rows, :b.hkv * b.d] = 0
        marks = sorted({j for m in range(0, n + block, block) for j in (m - 1, m) if 0 <= j < n} | ({n - 1} if n else set()))
        for i, j in enumerate(marks):
            for h in range(b.hkv):
                b.v[rows[j], h * b.d + (i + 29 * line) % b.d] = 1
    return b
