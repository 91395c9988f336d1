"""Trees of drafted tokens and plain fp64 forms of the operators over them, for the tests."""
import random

import torch

STEP = 2.0 ** -24                 # half a step of fp32, relative


def tree(k, seed, reach=4, nodes=None):
    """Parents of a tree of `nodes` nodes (default k) in k places."""
    r = random.Random(seed)
    m = k if nodes is None else nodes
    return [-1 if j == 0 else r.randrange(max(0, j - reach), j) if j < m else -2 for j in range(k)]


def path(row, j):
    """Places from the root to j; nothing where j, or a place on the way, holds no node."""
    out = []
    while j >= 0:
        if row[j] < -1 or row[j] >= j:
            return []
        out.append(j)
        j = row[j]
    return out[::-1]


def state_outputs(q, k, v, la, beta, S, row):
    """fp64 outputs [K, H, D] of a tree's nodes from the state S [H, D, D] by the recurrence itself, and a bound of the
    error that fp32 sums make in the operator's own order.

    The operator forms u_a = beta (v - S^T (A k) - sum_b m_ab u_b) and o = S^T (A q) + sum_a n_a u_a with m, n sums of D
    products.  With every term replaced by its magnitude (U, O), each level of the path adds at most the relative error
    of its sums (D + the path's length + a few, in half steps; products of alphas, expf's two steps each, another 6 a
    node), of what has come before."""
    K, H, D = q.shape
    out = torch.zeros(K, H, D, dtype=torch.float64)
    bound = torch.zeros(K, H, D, dtype=torch.float64)
    for h in range(H):
        S0 = S[h].double()
        after, U, alpha = {}, {}, {}
        for j in range(K):
            p = path(row, j)
            if not p:
                continue
            a = torch.ones(D, dtype=torch.float64) if la is None else torch.exp(la[j, h].double()).expand(D)
            alpha[j] = a
            kj, qj, vj, b = k[j, h].double(), q[j, h].double(), v[j, h].double(), beta[j, h].double()
            S1 = a[:, None] * (S0 if row[j] == -1 else after[row[j]])
            after[j] = S1 + b * torch.outer(kj, vj - S1.T @ kj)
            out[j, h] = after[j].T @ qj
            # magnitudes, along the path
            A = torch.ones(D, dtype=torch.float64)
            x, o = vj.abs(), torch.zeros(D, dtype=torch.float64)
            for c in reversed(p):
                kc = A * k[c, h].double().abs()
                if c != j:
                    x = x + (kj.abs() @ kc) * U[c]
                    o = o + (qj.abs() @ kc) * U[c]
                A = A * alpha[c]
            x = x + S0.abs().T @ (A * kj.abs())
            U[j] = b.abs() * x
            o = o + (qj.abs() @ kj.abs()) * U[j] + S0.abs().T @ (A * qj.abs())
            n = len(p)
            bound[j, h] = (n + 1) * (D + 8 * n + 16) * STEP * o * 1.01
    return out, bound
