"""The bf16 products, their gradients, combine's gradient and the dense product in 64 bits on the CPU,
with the error bounds the GPU results are held to. Written from the operators' definitions; nothing of
the library is used."""
import torch

from expert_reference import U16, U32

TINY = 2.0 ** -133        # a flush to bf16's subnormal step


def product64(x, w):
    """(x @ w, bound of its fp32 error): products of bf16 values are exact, and each of the n additions
    (and 8 more where partial sums meet) rounds every term once at most."""
    n = x.shape[-1]
    return x @ w, (n + 8) * U32 * (x.abs() @ w.abs())


def rounded(v, err):
    """Tolerance of a value within err of v, rounded once to bf16."""
    return err + U16 * (v.abs() + err) + TINY


def swiglu64(g, u, dg=0.0, du=0.0):
    """(h, bound): g and u are off by dg and du. |silu'| <= 1.1; the exponential's argument is rounded
    once (relative error 1.5 |g| half steps), the sum, reciprocal and products add 8."""
    silu = g * torch.sigmoid(g)
    h = silu * u
    err = 1.1 * dg * (u.abs() + du) + (silu.abs() + 1.1 * dg) * du
    return h, err + h.abs() * U32 * (8 + 3 * g.abs()) + 2.0 ** -120


def silu_grad64(g):
    s = torch.sigmoid(g)
    return s * (1 + g * (1 - s))


def swiglu_grad64(dh, ddh, g, u):
    """(dg, du, their bounds) for dh off by ddh. s is off by (1.5 |g| + 8) half steps of its value; 1 - s
    by a half step more, absolute, which g multiplies; each product rounds once."""
    s = torch.sigmoid(g)
    ds = s * U32 * (8 + 3 * g.abs())
    poly = 1 + g * (1 - s)
    dpoly = g.abs() * (ds + U32) + 2 * U32 * (1 + (g * (1 - s)).abs())
    a = dh * u
    dg, du = a * s * poly, dh * g * s
    eg = (ddh * u.abs()) * (s * poly.abs()) + a.abs() * (ds * poly.abs() + s * dpoly)
    eu = ddh * (g * s).abs() + dh.abs() * g.abs() * ds
    # second-order terms and the products' own roundings
    return (dg, du, 1.01 * eg + 6 * U32 * (dg.abs() + eg) + 2.0 ** -120,
            1.01 * eu + 4 * U32 * (du.abs() + eu) + 2.0 ** -120)


def act64(name, z):
    return {"none": lambda: z, "relu": lambda: z.clamp_min(0), "silu": lambda: z * torch.sigmoid(z),
            "gelu": lambda: z * torch.special.ndtr(z)}[name]()


def act_grad64(name, z):
    if name == "none":
        return torch.ones_like(z)
    if name == "relu":
        return (z > 0).double()
    if name == "silu":
        return silu_grad64(z)
    return torch.special.ndtr(z) + z * torch.exp(-z * z / 2) / (2 * torch.pi) ** 0.5


# Bounds of an activation's own evaluation in fp32, absolute. silu: as in swiglu64. gelu: z/2 * (1 + erf),
# erf within 16 half steps of 1 and 1 + erf rounded once: |z| * 17 half steps with the products.
def act_error(name, z):
    if name == "silu":
        return (z * torch.sigmoid(z)).abs() * U32 * (8 + 3 * z.abs()) + 2.0 ** -120
    if name == "gelu":
        return z.abs() * U32 * 17 + 2.0 ** -120
    return torch.zeros_like(z)


# silu': s within (8 + 3 |z|) half steps, the polynomial as in swiglu_grad64. gelu': erf as above;
# z exp(-z^2 / 2): the exponent's argument is rounded twice, z^2 half steps each at most, the rest 8.
def act_grad_error(name, z):
    if name == "silu":
        s = torch.sigmoid(z)
        ds = s * U32 * (8 + 3 * z.abs())
        poly = 1 + z * (1 - s)
        return (ds * poly.abs() + s * (z.abs() * (ds + U32) + 2 * U32 * (1 + (z * (1 - s)).abs()))
                + 4 * U32 + 2.0 ** -120)
    if name == "gelu":
        return U32 * (17 + z.abs() * torch.exp(-z * z / 2) * (8 + 2 * z * z)) + 2.0 ** -120
    return torch.zeros_like(z)
