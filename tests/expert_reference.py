"""The experts' operators in 64 bits on the CPU, with the error bounds the GPU results are held
to. Written from the operators' definitions; nothing of the library is used."""
import numpy as np
import torch

BLOCK = 128
U32 = 2.0 ** -24          # half a step of fp32
U16 = 2.0 ** -8           # half a step of bf16 (its eps / 2), relative to the value
U8 = 2.0 ** -4            # half a step of E4M3


def codes(rng, shape, scale=1.0):
    """Random E4M3 codes of N(0, scale) values."""
    v = torch.from_numpy(rng.standard_normal(shape, dtype=np.float32) * np.float32(scale))
    return v.clamp(-448, 448).to(torch.float8_e4m3fn)


def quantise(x):
    """E4M3 codes and fp32 scales (amax / 448) per row and 128 channels of fp32 rows."""
    b = x.unflatten(-1, (-1, BLOCK))
    s = b.abs().amax(-1) / 448
    return (b / s[..., None]).clamp(-448, 448).flatten(-2).to(torch.float8_e4m3fn), s


def weights64(w_q, w_scale):
    """[N, H] codes and [ceil(N/128), H/128] scales -> float64 values."""
    full = w_scale.double().repeat_interleave(BLOCK, 0)[:w_q.shape[0]].repeat_interleave(BLOCK, 1)
    return w_q.double() * full


def rows64(q, scale):
    return q.double() * scale.double().repeat_interleave(BLOCK, 1)


def product64(q, scale, w_q, w_scale):
    """(rows * weights^T, bound of its fp32 error).

    Each product of two codes is exact in fp32 (4 + 4 significant bits); a block's 127 additions,
    the product of the two scales, the fmaf and the running sum over the H/128 blocks each round
    once, so every term carries at most 128 + H/128 + 2 half steps."""
    x, w = rows64(q, scale), weights64(w_q, w_scale)
    return x @ w.T, (130 + x.shape[1] // BLOCK) * U32 * (x.abs() @ w.abs().T)


def fp8_product_error(q, scale, w_q, w_scale):
    """Bound of what the FP8 matrix instruction cuts off.

    It aligns the products of a group (at most 16 consecutive codes) to the largest exponent sum E
    in the group and keeps 13 binary places below it (pinned by test_matrix_instruction_alignment):
    a product loses less than 2^(E-13), and 2^E <= max|x| max|w| over the group, so a group of 16
    loses less than 16 * 2^-13 * max|x| * max|w|."""
    x, w = rows64(q, scale).abs(), weights64(w_q, w_scale).abs()
    group = lambda v: v.unflatten(1, (-1, 16)).amax(-1)  # noqa: E731
    return 16 * 2.0 ** -13 * (group(x) @ group(w).T)


def gemm_tolerance(y, err):
    """One rounding of a value within err of y to bf16 (smallest normal 2^-126, so a flush to a
    subnormal step is below 2^-133)."""
    return err + U16 * (y.abs() + err) + 2.0 ** -133


def swiglu64(q, scale, w_q, w_scale):
    """(h, bound of its fp32 error): |silu'| <= 1.1, |silu(g)| <= |g|; the exponential's argument
    is rounded once (relative error |g| * U32 * 1.5, with the hardware's own 2 half steps), and the
    sum, quotient and product add 4 more."""
    v, err = product64(q, scale, w_q, w_scale)
    (g, u), (dg, du) = v.chunk(2, 1), err.chunk(2, 1)
    silu = g * torch.sigmoid(g)
    h = silu * u
    dh = 1.1 * dg * (u.abs() + du) + (silu.abs() + 1.1 * dg) * du
    return h, dh + h.abs() * U32 * (8 + 3 * g.abs()) + 2.0 ** -120


def layer64(x, idx, w, w13, w2):
    """(out, tolerance) of a whole layer: x [T, H], idx and w [T, K], and per expert the float64
    weights w13(e) [2I, H] and w2(e) [H, I].

    fp32 sums of exact products: a sum of n terms rounds each at most n times (and the block
    scales and the wavefronts' meeting add at most 8). h is held as hi + lo, two bf16: |h - hi| <=
    U16 |h|, and lo is rounded to within U16 of that. The weighted sum rounds K times, out once."""
    T, H = x.shape
    out = torch.zeros(T, H, dtype=torch.float64)
    tol = torch.zeros(T, H, dtype=torch.float64)
    sums = torch.zeros(T, H, dtype=torch.float64)
    x = x.double()
    for e in sorted(set(idx.reshape(-1).tolist())):
        t, j = torch.nonzero(idx == e, as_tuple=True)
        a, b = w13(e), w2(e)
        if a is None:
            continue
        I = b.shape[1]
        v = x[t] @ a.T
        err = (H + 8) * U32 * (x[t].abs() @ a.abs().T)
        (g, u), (dg, du) = v.chunk(2, 1), err.chunk(2, 1)
        silu = g * torch.sigmoid(g)
        h = silu * u
        dh = 1.1 * dg * (u.abs() + du) + (silu.abs() + 1.1 * dg) * du
        dh = dh + h.abs() * U32 * (8 + 3 * g.abs()) + 2.0 ** -120
        dh = dh + U16 * U16 * (h.abs() + dh)
        y = h @ b.T
        dy = dh @ b.abs().T + (2 * I + 8) * U32 * ((h.abs() + dh) @ b.abs().T)
        wt = w[t, j].double()[:, None]
        out.index_add_(0, t, wt * y)
        tol.index_add_(0, t, wt.abs() * dy)
        sums.index_add_(0, t, wt.abs() * (y.abs() + dy))
    tol += idx.shape[1] * U32 * sums
    return out, tol + U16 * (out.abs() + tol) + 2.0 ** -133
