"""Combine's gradient, the dense product with its epilogue and its gradients against the definitions
in 64 bits."""
import numpy as np
import pytest
import torch

from combine_ep_layout_06_amd import binding as B

import product_reference as P
from expert_reference import U32

pytestmark = pytest.mark.gpu

DEV = "cuda"
SENTINEL = 0x5A5A
BF16 = torch.bfloat16


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    B.load_library()


def randn(rng, *shape, scale=1.0):
    return torch.from_numpy(rng.standard_normal(shape, dtype=np.float32) * np.float32(scale)).to(BF16)


def sentinel(*shape):
    return torch.full(shape, SENTINEL, dtype=torch.int16, device=DEV).view(BF16)


def close(got, want, tol, what):
    bad = ~((got - want).abs() <= tol)
    assert not bad.any(), (what, int(bad.sum()), float((got - want).abs().max()), float(tol.max()))


# T, H, E, K, C: one pair; odd widths; drops; K above a wavefront's pairs; rows longer than one pass; the
# last two with a wavefront for each pair
COMBINE = [(1, 8, 1, 1, 1), (7, 72, 4, 3, 3), (65, 512, 16, 4, 9), (33, 1032, 128, 8, 33),
           (5, 4104, 40, 33, 5), (129, 2056, 8, 2, 40), (1500, 264, 12, 6, 500),
           (1100, 2056, 16, 8, 700)]


@pytest.mark.parametrize("T,H,E,K,C", COMBINE)
@pytest.mark.parametrize("packed", [False, True])
def test_combine_grad(T, H, E, K, C, packed):
    print(f"[combine_grad] T={T} H={H} E={E} K={K} C={C} packed={packed}", flush=True)
    rng = np.random.default_rng(T * H + packed)
    idx = torch.from_numpy(rng.integers(-1, E + 1, size=(T, K)).astype(np.int32))   # -1 and E too
    idx_d = idx.to(DEV)
    if packed:
        lay = B.ep_layout_packed(idx_d, E, C, 1, 16)
        first = lay["packed_offset"].cpu().long()
        rows = int(first[-1]) + 3
    else:
        lay = B.ep_layout(idx_d, E, C, 1)
        first = torch.arange(E + 1) * C
        rows = E * C
    slot = lay["slot"].cpu()
    dout, w = randn(rng, T, H), torch.from_numpy(rng.standard_normal((T, K)).astype(np.float32))
    y = randn(rng, rows, H)
    kept = slot >= 0
    row = torch.where(kept, first[idx.long().clamp(0, E - 1)] + slot, 0)
    held = torch.zeros(rows, dtype=torch.bool)
    held[row[kept]] = True
    y[~held] = float("nan")
    dy, dw = sentinel(rows, H), torch.full((T, K), float("nan"), device=DEV)
    if packed:
        B.ep_combine_grad_packed(dout.to(DEV), y.to(DEV), idx_d, lay["slot"], lay["packed_offset"],
                                 w.to(DEV), E, C, dy=dy, dtopk_w=dw)
    else:
        B.ep_combine_grad(dout.to(DEV), y.view(E, C, H).to(DEV), idx_d, lay["slot"], w.to(DEV), C,
                          dy=dy.view(E, C, H), dtopk_w=dw)
    got, dw = dy.cpu(), dw.cpu().double()
    assert (got[~held].view(torch.int16) == SENTINEL).all(), "a row that holds no pair was written"
    assert (dw[~kept] == 0).all()
    t, j = torch.nonzero(kept, as_tuple=True)
    d, v = dout[t].double(), y[row[t, j]].double()
    want = w[t, j].double()[:, None] * d
    close(got[row[t, j]].double(), want, P.rounded(want, U32 * want.abs()), "dy")
    close(dw[t, j], (d * v).sum(1), (H + 8) * U32 * (d * v).abs().sum(1), "dw")


LINEAR = [(1, 8, 8), (1, 4096, 520), (3, 264, 72), (17, 72, 136), (64, 512, 256), (130, 200, 1032),
          (300, 1096, 264), (513, 64, 8), (2100, 136, 520), (20000, 520, 8)]


def linear_inputs(T, H, N):
    rng = np.random.default_rng(T + H + N)
    return rng, randn(rng, T, H), randn(rng, N, H, scale=2 * H ** -0.5)


@pytest.mark.parametrize("T,H,N", LINEAR)
@pytest.mark.parametrize("act,bias,residual,keep", [
    ("none", False, False, False), ("none", True, True, False), ("relu", True, False, True),
    ("silu", False, True, True), ("gelu", True, True, False)])
def test_linear(T, H, N, act, bias, residual, keep):
    print(f"[linear] T={T} H={H} N={N} {act} {bias} {residual} {keep}", flush=True)
    rng, x, w = linear_inputs(T, H, N)
    b = randn(rng, N) if bias else None
    r = randn(rng, T, N) if residual else None
    out, pre = sentinel(T, N), sentinel(T, N) if keep else None
    on = lambda t: None if t is None else t.to(DEV)  # noqa: E731
    if residual and act == "gelu":             # in place
        out.copy_(r)
        res = out
    else:
        res = on(r)
    B.ep_linear(x.to(DEV), w.to(DEV), bias=on(b), act=act, residual=res, pre=pre, out=out)
    z, err = P.product64(x.double(), w.double().T)
    if bias:
        z = z + b.double()
        err = err + U32 * (z.abs() + err)
    if keep:
        close(pre.cpu().double(), z, P.rounded(z, err), "pre")
    want = P.act64(act, z)
    # |act'| <= 1.13 for each of them
    err = 1.13 * err + P.act_error(act, z) + 3 * U32 * (want.abs() + 1.13 * err)
    if residual:
        want = want + r.double()
        err = err + U32 * (want.abs() + err)
    close(out.cpu().double(), want, P.rounded(want, err), "out")


@pytest.mark.parametrize("T,H,N", LINEAR)
@pytest.mark.parametrize("act", ["none", "relu", "silu", "gelu"])
def test_linear_grad(T, H, N, act):
    print(f"[linear_grad] T={T} H={H} N={N} {act}", flush=True)
    rng, x, w = linear_inputs(T, H, N)
    dout = randn(rng, T, N)
    pre = None if act == "none" else randn(rng, T, N, scale=2)
    dx, dw, dbias = B.ep_linear_grad(dout.to(DEV), x.to(DEV), w.to(DEV), act=act,
                                     pre=None if pre is None else pre.to(DEV))
    dz = dout.double()
    err = torch.zeros_like(dz)
    if pre is not None:
        p = pre.double()
        dz, d = dz * P.act_grad64(act, p), dz
        err = d.abs() * P.act_grad_error(act, p) + U32 * dz.abs()
    close(dbias.cpu().double(), dz.sum(0), err.sum(0) + (T + 8) * U32 * (dz.abs() + err).sum(0),
          "dbias")
    # the products' operand is dz rounded to bf16
    op = P.rounded(dz, err) if pre is not None else torch.zeros_like(dz)
    top = dz.abs() + op
    want = dz @ w.double()
    tol = op @ w.double().abs() + (N + 8) * U32 * (top @ w.double().abs())
    close(dx.cpu().double(), want, P.rounded(want, tol), "dx")
    want = dz.T @ x.double()
    tol = op.T @ x.double().abs() + (T + 8) * U32 * (top.T @ x.double().abs())
    close(dw.cpu().double(), want, P.rounded(want, tol), "dw")


def test_combine_grad_of_more_pairs_than_a_grid_row_holds():
    """A wavefront for each of 67.2 million pairs is more than 2^32 threads."""
    T, H, K = 8_400_000, 8, 8
    g = torch.Generator(device=DEV)
    g.manual_seed(6)
    dout = torch.randn(T, H, generator=g, device=DEV).to(BF16)
    w = torch.randn(T, K, generator=g, device=DEV)
    y = torch.randn(K, T, H, generator=g, device=DEV).to(BF16)
    idx = torch.arange(K, dtype=torch.int32, device=DEV).repeat(T, 1)
    slot = torch.arange(T, dtype=torch.int32, device=DEV)[:, None].repeat(1, K)
    drop = torch.rand(T, K, generator=g, device=DEV) < 0.05
    slot[drop] = -1
    dy = torch.full((K, T, H), SENTINEL, dtype=torch.int16, device=DEV).view(BF16)
    dw = torch.full((T, K), float("nan"), device=DEV)
    print("[combine_grad]", T * K, "pairs", flush=True)
    B.ep_combine_grad(dout, y, idx, slot, w, T, dy=dy, dtopk_w=dw)
    for j in range(K):
        d, v = dout.double(), y[j].double()
        want = w[:, j].double()[:, None] * d
        got = dy[j].double()
        off = (got - want).abs() - P.rounded(want, U32 * want.abs())
        assert (off[~drop[:, j]] <= 0).all(), j
        assert (dy[j].view(torch.int16)[drop[:, j]] == SENTINEL).all(), j
        off = (dw[:, j].double() - (d * v).sum(1)).abs() - (H + 8) * U32 * (d * v).abs().sum(1)
        assert (off[~drop[:, j]] <= 0).all() and (dw[:, j][drop[:, j]] == 0).all(), j
