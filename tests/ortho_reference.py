"""Newton-Schulz steps in 64 bits on the CPU, and a model of what fp16 operands
do to them: the roundings of the kernels' number formats at their places, all
else in 64 bits."""
import torch

D, F = torch.float64, torch.float32
JORDAN = (3.4445, -4.7750, 2.0315)


def coefficients(steps, coef=JORDAN):
    """The fp32 values a call passes, one triple a step."""
    each = [coef] * steps if not hasattr(coef[0], "__len__") else list(coef)
    return [[float(torch.tensor(v, dtype=F)) for v in c] for c in each]


def start(x, eps):
    x = x.to(D)
    size = x.norm() + float(torch.tensor(eps, dtype=F))
    return x / size if size > 0 else x * 0


def exact(x, steps=5, coef=JORDAN, eps=1e-7):
    x = start(x, eps)
    for a, b, c in coefficients(steps, coef):
        if x.shape[0] <= x.shape[1]:
            g = x @ x.T
            x = a * x + b * (g @ x) + c * (g @ (g @ x))
        else:
            g = x.T @ x
            x = a * x + b * (x @ g) + c * ((x @ g) @ g)
    return x


def half(v, scale):
    return (v * scale).to(torch.float16).to(D) / scale


def model(x, steps=5, coef=JORDAN, eps=1e-7):
    """X in two fp16 numbers of which products read the first, off-diagonals of
    both symmetric matrices in fp16, their diagonals apart."""
    x = start(x, eps)
    tall = x.shape[0] > x.shape[1]
    x = x.T if tall else x
    for a, b, c in coefficients(steps, coef):
        hi = half(x, 4096.0)
        x = hi + half(x - hi, 4096.0)
        g = hi @ hi.T
        d = g.diagonal().clone()
        o = half(g - torch.diag(d), 256.0)
        s = o @ o
        p = b * o + c * (s + (d[:, None] + d[None]) * o)
        dp = b * d + c * (s.diagonal() + d * d)
        p = half(p - torch.diag(p.diagonal()), 64.0)
        x = (a + dp)[:, None] * x + p @ hi
    x = half(x, 4096.0)
    return x.T if tall else x


def allowance(x, steps=5, coef=JORDAN, eps=1e-7):
    """(exact result, bound on a kernel's distance from it in 2-norm): the kernel rounds where the model does, to numbers that its fp32 sums (2e-6 at any length used
    here) may turn to the neighbour, so its error is another draw of the same roundings: three times the model's, which for the few roundings of a small matrix
    leaves room for the worst signs."""
    e = exact(x, steps, coef, eps)
    return e, 3 * (model(x, steps, coef, eps) - e).norm() + 1e-5 * e.norm()
