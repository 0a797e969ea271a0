"""Plain 64-bit forms of the hybrid target's operators, and how far their kernels may be off."""
import math

import torch

B8, E24, S16 = 2.0 ** -8, 2.0 ** -24, 2.0 ** -16
BIG = 64                    # tokens that the kernels take at a time


def tree(r, n, reach=12, roots=1):
    """Parents of a random tree in drafting order; the first `roots` nodes have none."""
    return [-1] * min(roots, n) + [r.randint(max(0, i - reach), i - 1) for i in range(roots, n)]


def ancestors(parents):
    """Sets of places: of each node, the nodes on its path, without itself."""
    out = []
    for i, p in enumerate(parents):
        out.append(set() if p < 0 else out[p] | {p})
    return out


def mask_of(parents, words=1):
    """int64 [n, words] as the operators take it: ancestors and the node itself."""
    rows = []
    for i, up in enumerate(ancestors(parents)):
        bits = [0] * words
        for j in up | {i}:
            if j // 64 < words:
                bits[j // 64] |= 1 << (j % 64)
        rows.append([b - (1 << 64) if b >> 63 else b for b in bits])
    return torch.tensor(rows, dtype=torch.int64).view(-1, words)


def delta_steps(q, k, v, g, beta, s0, scale, l2, eps, parents=None):
    """The recurrence itself, of one head: q, k [n, dk], v [n, dv], s0 [dk, dv], all float64.  Outputs, last state."""
    if l2:
        q, k = (x / torch.sqrt((x * x).sum(1, keepdim=True) + eps) for x in (q, k))
    n = k.shape[0]
    states, out = [], torch.zeros(n, v.shape[1], dtype=torch.float64)
    for i in range(n):
        p = i - 1 if parents is None else parents[i]
        s = (s0 if p < 0 else states[p]) * math.exp(g[i])
        s = s + torch.outer(k[i], beta[i] * (v[i] - s.t() @ k[i]))
        out[i] = scale * (s.t() @ q[i])
        states.append(s)
    return out, states[-1] if n else s0


def delta_bounds(q, k, v, g, beta, s0, scale, l2, eps, parents=None):
    """Bounds of the errors of delta_steps' outputs [n, dv] and last state [dv] (every element of a column).

    The kernels take 64 tokens at a time: R = beta (V - e^G K S), U = T R with T the inverse of the triangular system,
    S' = e^G S + (e^.. K)^T U, out = scale (e^G Q S + P U).  What is FP32 goes into the products as two BF16 values (off by
    2^-16) or, for out, as one (2^-8); sums of n products are off by n 2^-23 of the sum of magnitudes (matrix instructions may
    cut off); norms, exponentials and factors of them by 16 roundings and what G's rounding to FP32 makes of it.
    An error of a state's column lives on with no larger norm (each token's step is a contraction where beta |k|^2 <= 2 and
    g <= 0), and an error of R at token t is as one of v there: it reaches the state with the norm |k_t| of its own."""
    if l2:
        q, k = (x / torch.sqrt((x * x).sum(1, keepdim=True) + eps) for x in (q, k))
    n, dk = k.shape
    few = 16 * E24
    sums = 2 * (dk + BIG) * E24
    err_s = torch.zeros(v.shape[1], dtype=torch.float64)      # the column norms of the state's error
    out = torch.zeros(n, v.shape[1], dtype=torch.float64)
    s = s0
    step = n if parents is not None else BIG
    for c in range(0, n, step or 1):
        qc, kc, vc, gc, bc = (x[c:c + step] for x in (q, k, v, g, beta))
        m = kc.shape[0]
        if parents is None:
            before = torch.ones(m, m, dtype=torch.bool).tril(-1)
        else:
            before = torch.zeros(m, m, dtype=torch.bool)
            for i, up in enumerate(ancestors(parents)):
                before[i, sorted(up)] = True
        own = before | torch.eye(m, dtype=torch.bool)
        total = own.double() @ gc
        decay = torch.exp(torch.where(own, total[:, None] - total[None], torch.tensor(0.0)).clamp(max=80))
        gk = (kc @ kc.t()) * decay
        a = torch.where(before, bc[:, None] * gk, torch.tensor(0.0, dtype=torch.float64))
        t = torch.linalg.solve_triangular(a + torch.eye(m, dtype=torch.float64), torch.eye(m, dtype=torch.float64), upper=False)
        p = torch.where(own, scale * decay * (qc @ kc.t()), torch.tensor(0.0, dtype=torch.float64))
        grown = torch.exp(total)[:, None]
        ks = kc.abs() @ s.abs()
        r = bc[:, None] * (vc - grown * (kc @ s))
        r_abs = bc[:, None].abs() * (vc.abs() + grown * ks)
        u = t @ r
        knorm = kc.norm(dim=1)[:, None]
        # R: what the split of S and the sums do, and the state's own error
        dr_new = (S16 + sums + few) * r_abs
        dr = dr_new + bc[:, None].abs() * grown * knorm * err_s
        # U: T and R as two values each, T's own making (errors of the factors a, and of substitution, both through T), the sums
        t_abs = t.abs()
        dt = t_abs @ ((sums + few) * a.abs()) @ t_abs
        du_new = (2 * S16 + sums + few) * (t_abs @ r.abs()) + dt @ r.abs()
        du = t_abs @ dr + du_new
        # out
        qs = scale * abs(1.0) * grown * (qc.abs() @ s.abs())
        pu = p.abs() @ u.abs()
        o = scale * grown * (qc @ s) + p @ u
        out[c:c + m] = (B8 * o.abs() + 1.02 * B8 * qs + 2.04 * B8 * pu + (sums + few) * (qs + pu) + p.abs() @ du +
                        abs(scale) * grown * qc.norm(dim=1)[:, None] * err_s)
        left = torch.exp((total[-1] - total).clamp(max=80))[:, None]
        if parents is None:
            err_s = (math.exp(total[-1]) * err_s + (left * knorm * (dr_new + du_new)).sum(0) +
                     (S16 + sums + few) * ((left * knorm * u.abs()).sum(0) + math.exp(total[-1]) * s.norm(dim=0)))
            s = math.exp(total[-1]) * s + (left * kc).t() @ u
    return out * 1.01 + 1e-30, err_s * 1.01 + 1e-30


def conv_ref(x, weight, bias, past, silu, parents=None):
    """x [n, c], past [w - 1, c], all float64 -> y, the sum of magnitudes behind it, the new past."""
    w = weight.shape[1]
    line = torch.cat((past, x))
    y = torch.zeros_like(x) + (0 if bias is None else bias)
    mag = y.abs()
    for i in range(x.shape[0]):
        at = i
        for back in range(w):
            y[i] += weight[:, w - 1 - back] * line[w - 1 + at]
            mag[i] += (weight[:, w - 1 - back] * line[w - 1 + at]).abs()
            at = at - 1 if at < 0 or parents is None else parents[at]
    return (y / (1 + torch.exp(-y)) if silu else y), mag, line[x.shape[0]:]


def verify_ref(logits, tokens, u, parents, temp, q=None, accept_u=None):
    """One request: logits [n, v], parents with node 0 first -> accepted nodes, the token that follows."""
    n, v = logits.shape

    def law(i):
        z = logits[i].double()
        z = torch.where(z.isnan(), -math.inf, z)
        top = z.max()
        if top == -math.inf:
            return None
        if not temp > 0 or top == math.inf:
            p = torch.zeros(v, dtype=torch.float64)
            p[int((z == top).nonzero()[0])] = 1
            return p
        return torch.exp((z - top) / temp)          # not divided by the sum: borders between tokens stay where they are

    def take(w, x):
        if w is None:
            return -1
        x = min(max(x, 0.0), 1 - 2.0 ** -24) if x == x else 0.0
        edges = w.cumsum(0)
        i = int((edges <= x * edges[-1]).sum())
        return min(i, int(w.nonzero()[-1]))

    at, found = 0, [0]
    while True:
        w = law(at)
        p = None if w is None else w / w.sum()
        kids = [i for i in range(1, n) if parents[i] == at]
        if q is None:
            got = take(w, float(u[at]))
            kids = [i for i in kids if int(tokens[i]) == got and got >= 0]
            if not kids:
                return found, got
        else:
            if not kids:
                return found, take(w, float(u[at]))
            i, x = kids[0], int(tokens[kids[0]])
            a = float(accept_u[i])
            a = min(max(a, 0.0), 1 - 2.0 ** -24) if a == a else 0.0
            if not (0 <= x < v and p is not None and a * float(q[i, x]) < float(p[x])):
                if p is None:
                    return found, -1
                rest = (p - q[i].double()).clamp(min=0).nan_to_num(0.0)
                return found, take(rest if float(rest.sum()) > 0 else w, float(u[at]))
        at = kids[0]
        found.append(at)
