"""Float64 forms of the layer operators with a bound on what the kernels may
differ from them.

A value travels as (v, e): the float64 value from the same inputs, and a bound
on the kernel's error in it.  The bounds follow the kernels' arithmetic:

* a product of 16-bit operands is exact in FP32; the tensor cores add 16
  products at a time to an FP32 accumulator and may truncate, so a sum of K
  terms is within (K / 16 + 16) 2^-22 of the sum of magnitudes (split sums add
  a few more roundings, covered by the 16);
* one rounding to BF16 (8 significant bits) is within 2^-8 of the value, to
  FP16 (11) within 2^-11, or half the smallest subnormal;
* FP32 steps and the activations' functions are within 2^-20 of the value.
"""

import math

import torch

F32 = 2.0 ** -20
ROUND = {torch.bfloat16: (2.0 ** -8, 0.0), torch.float16: (2.0 ** -11, 2.0 ** -25),
         torch.float32: (2.0 ** -24, 0.0)}
# largest |act'| and |act''|, rounded up
SLOPE = {"none": (1, 0), "relu": (1, 0), "gelu": (1.13, 0.8), "gelu_tanh": (1.13, 0.8),
         "silu": (1.1, 0.5), "sigmoid": (0.25, 0.1)}


def sum_bound(k):
    return (k / 16 + 16) * 2.0 ** -22


def exact(t):
    v = t.double()
    return v, torch.zeros_like(v)


def rounded(x, dtype):
    rel, least = ROUND[dtype]
    v, e = x
    return v, e + rel * (v.abs() + e) * 1.01 + least


def matmul(a, b):
    (av, ae), (bv, be) = a, b
    mag = (av.abs() + ae) @ (bv.abs() + be)
    return av @ bv, sum_bound(av.shape[1]) * mag + ae @ (bv.abs() + be) + av.abs() @ be


def t(x):
    return x[0].t(), x[1].t()


def add(a, b):
    v = a[0] + b[0]
    return v, a[1] + b[1] + F32 * v.abs()


def mul(a, b):
    v = a[0] * b[0]
    return v, a[1] * (b[0].abs() + b[1]) + a[0].abs() * b[1] + F32 * v.abs()


def act(name, z):
    """act(z) and act'(z)."""
    v, e = z
    if name == "none":
        return z, (torch.ones_like(v), torch.zeros_like(v))
    if name == "relu":
        # within the error of zero the slope is either
        return (v.clamp(min=0), e), ((v > 0).double(), (v.abs() <= e).double() * (e > 0))
    s1, s2 = SLOPE[name]
    if name in ("sigmoid", "silu"):
        s = torch.sigmoid(v)
        a, d = (s, s * (1 - s)) if name == "sigmoid" else (v * s, s * (1 + v * (1 - s)))
    elif name == "gelu":
        c = 0.5 * torch.erfc(-v / math.sqrt(2))
        a, d = v * c, c + v * torch.exp(-v * v / 2) / math.sqrt(2 * math.pi)
    else:
        s = torch.sigmoid(2 * math.sqrt(2 / math.pi) * (v + 0.044715 * v ** 3))
        a = v * s
        d = s + v * s * (1 - s) * 2 * math.sqrt(2 / math.pi) * (1 + 3 * 0.044715 * v * v)
    # FP32 evaluation: 2^-20 of the value's parts (|v| + 1 bounds their size)
    f = F32 * (1 + v.abs())
    return (a, s1 * e + f * torch.minimum(a.abs() + 2.0 ** -10, torch.ones_like(a) + v.abs())), \
           (d, s2 * e + f)


def linear(x, W, bias, residual, name, dt, out_dt=None):
    z = matmul(exact(x), exact(W))
    if bias is not None:
        z = add(z, exact(bias))
    y = act(name, z)[0]
    if residual is not None:
        y = add(y, exact(residual))
    return rounded(y, out_dt or dt), z


def column_sum(x):
    v, e = x
    return v.sum(0), e.sum(0) + v.shape[0] * 2.0 ** -24 * v.abs().sum(0)


def linear_grads(x, W, z, dout, name, dt):
    dz = mul(exact(dout), act(name, z)[1]) if name != "none" else exact(dout)
    dz16 = rounded(dz, dt) if name != "none" else dz
    return {"dx": rounded(matmul(dz16, t(exact(W))), dt),
            "dW": rounded(matmul(t(exact(x)), dz16), dt),
            "dbias": rounded(column_sum(dz), dt)}


def gated(x, Wg, Wu, Wd, residual, name, dt):
    g, u = matmul(exact(x), exact(Wg)), matmul(exact(x), exact(Wu))
    h = rounded(mul(act(name, g)[0], u), dt)
    y = matmul(h, exact(Wd))
    if residual is not None:
        y = add(y, exact(residual))
    return rounded(y, dt), (g, u, h)


def gated_grads(x, Wg, Wu, Wd, kept, dout, name, dt):
    g, u, h = kept
    dh = matmul(exact(dout), t(exact(Wd)))
    a, d = act(name, g)
    dg, du = rounded(mul(mul(dh, u), d), dt), rounded(mul(dh, a), dt)
    xt = t(exact(x))
    return {"dx": rounded(add(matmul(dg, t(exact(Wg))), matmul(du, t(exact(Wu)))), dt),
            "dW_gate": rounded(matmul(xt, dg), dt), "dW_up": rounded(matmul(xt, du), dt),
            "dW_down": rounded(matmul(t(h), exact(dout)), dt)}


def worst(got, ref):
    """The largest error over its bound (at most 1 where the kernel is right);
    where the reference is NaN or infinite the value has to be the same."""
    v, e = ref
    g = got.double()
    fine = torch.isfinite(v) & torch.isfinite(e)
    same = (torch.isnan(g) & torch.isnan(v)) | (g == v) | fine
    if not bool(same.all()):
        return math.inf
    if not bool(fine.any()):
        return 0.0
    r = (g - v).abs()[fine] / (e[fine] + 1e-300)
    r = torch.where((g - v).abs()[fine] == 0, torch.zeros_like(r), r)
    return float("inf") if bool(torch.isnan(r).any()) else float(r.max())
