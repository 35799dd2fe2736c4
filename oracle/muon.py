"""Newton-Schulz orthogonalisation and the momentum step with it, in float64
(K. Jordan et al., "Muon: An optimizer for hidden layers in neural networks",
2024), straight from the iteration on the matrix itself."""

import numpy as np

COEF = (3.4445, -4.7750, 2.0315)


def orthogonalize(u, steps=5, coef=COEF, eps=1e-7):
    u = u.astype(np.float64)
    x = u if u.shape[0] <= u.shape[1] else u.T
    x = x / (np.sqrt((x * x).sum()) + eps)
    a, b, c = coef
    for _ in range(steps):
        g = x @ x.T
        x = a * x + (b * g + c * (g @ g)) @ x
    return x if u.shape[0] <= u.shape[1] else x.T


def momentum(g, m, mu, grad_scale=1.0, nesterov=True):
    """(new momentum, update direction) in float32, each operation rounded."""
    f = np.float32
    g = (g.astype(f) * f(grad_scale)).astype(f)
    m = ((f(mu) * m.astype(f)).astype(f) + g).astype(f)
    return m, (g + (f(mu) * m).astype(f)).astype(f) if nesterov else m


def step(p, g, m, lr, mu, weight_decay=0.0, grad_scale=1.0, nesterov=True, steps=5, coef=COEF,
         eps=1e-7):
    """(p before its rounding, m): p in float64 from the float32 update."""
    m, u = momentum(g, m, mu, grad_scale, nesterov)
    s = np.sqrt(max(1.0, p.shape[0] / p.shape[1]))
    o = orthogonalize(u, steps, coef, eps)
    return p.astype(np.float64) * (1 - lr * weight_decay) - lr * s * o, m
