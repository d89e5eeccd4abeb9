"""Plain fp64 CPU oracle of the gated linear recurrence (test infrastructure only).

    a_t = exp(g_t),  h_t = a_t h_{t-1} + b_t x_t,  o_t = h_t,
    b_t = 1, 1 - a_t or sqrt(max(0, 1 - a_t^2)),

per sequence and channel, token by token, and its reverse-mode gradient.  Next
to each value stands a bound on what fp32 arithmetic may differ by.  Every
product chain of the recurrence is rounded a fixed number of times per token:
exp and the input's weight within C_EL of their values, and one product and one
fma each at most 2^-24 off, so a value that is a sum of terms with magnitudes
M accumulates, per token that its terms pass, at most C_STEP of M:

    M_t = a_t M_{t-1} + |b_t x_t|,      E_t = a_t E_{t-1} + C_STEP (a_t M_{t-1} + |b_t x_t|)

and the gradient's chain likewise.
"""

import numpy as np

C_EL = 2.0 ** -22    # exp: 2 ulp; sqrt(-expm1(2 g)): half of expm1's 2 ulp plus the root's
C_STEP = C_EL + 4 * 2.0 ** -24   # and the roundings of a product, a fma and one chunk join


def gates(g, gate):
    """a, b and b' = db/dg in fp64."""
    with np.errstate(divide="ignore", invalid="ignore"):
        a = np.exp(g)
        if gate == "none":
            return a, np.ones_like(a), np.zeros_like(a)
        if gate == "complement":
            return a, -np.expm1(g), -a
        b = np.sqrt(np.maximum(-np.expm1(2 * g), 0))
        return a, b, np.where(b > 0, -a * a / np.where(b > 0, b, 1), 0)


def lru_fwd(x, g, cu, gate, h0=None):
    """(o [T, D], hT [N, D], bound of o, bound of hT)."""
    T, D = x.shape
    N = len(cu) - 1
    a, b, _ = gates(g, gate)
    u = b * x
    o, eo = np.zeros((T, D)), np.zeros((T, D))
    hT, eT = np.zeros((N, D)), np.zeros((N, D))
    for n in range(N):
        h = np.zeros(D) if h0 is None else h0[n].copy()
        m, e = np.abs(h), np.zeros(D)
        for t in range(cu[n], cu[n + 1]):
            e = a[t] * e + C_STEP * (a[t] * m + np.abs(u[t]))
            m = a[t] * m + np.abs(u[t])
            h = a[t] * h + u[t]
            o[t], eo[t] = h, e
        hT[n], eT[n] = h, e
    return o, hT, eo, eT


def lru_bwd(x, g, cu, gate, dO, h0=None, dhT=None):
    """dict of gradients dx, dg, dh0 and dict of their bounds."""
    T, D = x.shape
    N = len(cu) - 1
    a, b, db = gates(g, gate)
    o, _, eo, _ = lru_fwd(x, g, cu, gate, h0)
    big, _, _, _ = lru_fwd(np.abs(x), g, cu, gate, None if h0 is None else np.abs(h0))
    r = dict(dx=np.zeros((T, D)), dg=np.zeros((T, D)), dh0=np.zeros((N, D)))
    bound = {k: np.zeros_like(v) for k, v in r.items()}
    for n in range(N):
        k = np.zeros(D) if dhT is None else dhT[n].copy()
        m, e = np.abs(k), np.zeros(D)
        first = np.zeros(D) if h0 is None else h0[n]
        for t in range(cu[n + 1] - 1, cu[n] - 1, -1):
            d = k + dO[t]
            md = m + np.abs(dO[t])
            ed = e + 2.0 ** -24 * md
            hp = o[t - 1] if t > cu[n] else first
            mp = big[t - 1] if t > cu[n] else np.abs(first)
            ep = eo[t - 1] if t > cu[n] else np.zeros(D)
            r["dx"][t] = b[t] * d
            bound["dx"][t] = b[t] * (ed + 2 * C_EL * md)
            r["dg"][t] = d * (a[t] * hp + db[t] * x[t])
            size = a[t] * mp + np.abs(db[t] * x[t])
            bound["dg"][t] = ed * size + md * (a[t] * ep + 4 * C_STEP * size)
            k = a[t] * d
            e = a[t] * ed + C_STEP * a[t] * md
            m = a[t] * md
        r["dh0"][n], bound["dh0"][n] = k, e
    return r, bound
