"""Plain 64-bit forms of the training pass's operators: the gradients of combine
and dispatch, the bf16 expert products and theirs.

A float sum of n products off by at most SUM(n) times the sum of their
magnitudes: the matrix instruction adds 32 products, each addition off by one
unit in the last place at most (it may cut off instead of rounding), and the
instructions' results follow one another."""

from __future__ import annotations

import torch

U32 = 2.0 ** -24
U_BF16 = 2.0 ** -8
TINY = 2.0 ** -133          # the least bf16


def SUM(n):
    return (n / 32 + 34) * 2 * U32


def bf16_tol(want, off):
    """A value off by `off` and then rounded."""
    return want.abs() * U_BF16 * (1 + U32) + off * (1 + U_BF16) + TINY


def rows_of(T, E, R, k, idx, ll):
    """Slots of a layout ([T,R] or, per expert, [T,k], -1 without a row) and their
    number, by the definition, on the CPU."""
    idx = idx.cpu().tolist()
    n = 0
    if ll:
        slot = [[-1] * k for _ in range(T)]
        for e in range(E):
            for t in range(T):
                for j in range(k):
                    if idx[t][j] == e:
                        slot[t][j] = n
                        n += 1
    else:
        slot = [[-1] * R for _ in range(T)]
        for r in range(R):
            for t in range(T):
                if any(0 <= e < E and e // (E // R) == r for e in idx[t]):
                    slot[t][r] = n
                    n += 1
    return torch.tensor(slot, dtype=torch.int32).view(T, k if ll else R), n


def served(T, E, R, k, idx, slot, ll):
    """(t, row, choices that the row serves), over all rows."""
    idx, slot = idx.cpu().tolist(), slot.cpu().tolist()
    for t in range(T):
        for i in range(k if ll else R):
            s = slot[t][i]
            if s >= 0:
                yield t, s, [i] if ll else [j for j in range(k) if 0 <= idx[t][j] < E and idx[t][j] // (E // R) == i]


def spread(sizes, M, first=0):
    """Offsets of groups of these sizes from row `first` on."""
    off = [first]
    for n in sizes:
        off.append(off[-1] + n)
    assert off[-1] <= M
    return torch.tensor(off, dtype=torch.int32, device="cuda")


def product64(rows, off, w):
    """[M, N] in 64 bits and the sums of the magnitudes; rows of no expert zero."""
    off = off.tolist()
    out = torch.zeros(rows.shape[0], w.shape[1], dtype=torch.float64, device="cuda")
    mag = torch.zeros_like(out)
    for g in range(len(off) - 1):
        a, b = off[g], off[g + 1]
        if a < b:
            x, v = rows[a:b].double(), w[g].double().t().contiguous()
            out[a:b] = x @ v
            mag[a:b] = x.abs() @ v.abs()
    return out, mag


def weights64(rows, off, grad_out):
    """Gradient of the weights [G, N, K] in 64 bits and the sums of the magnitudes."""
    off = off.tolist()
    G = len(off) - 1
    out = torch.zeros(G, grad_out.shape[1], rows.shape[1], dtype=torch.float64, device="cuda")
    mag = torch.zeros_like(out)
    for g in range(G):
        a, b = off[g], off[g + 1]
        if a < b:
            d, x = grad_out[a:b].double().t().contiguous(), rows[a:b].double()
            out[g] = d @ x
            mag[g] = d.abs() @ x.abs()
    return out, mag
