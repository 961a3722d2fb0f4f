"""The bf16 products and the dense product's gradients at the edges of what their documentation allows:
widths just below 2^20, the most rows of ep_linear_grad, subnormal and huge values."""
import pytest
import torch

from combine_ep_layout_06_amd import binding as B

import product_reference as P
from expert_reference import U32
from test_gpu_gradients import close
from test_gpu_products import kernels

pytestmark = pytest.mark.gpu

DEV = "cuda"
BF16 = torch.bfloat16
WIDE, NARROW = 2 ** 20 - 8, 1016      # their product is 2^30 less 1.4%


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    B.load_library()


def generator(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return g


def normal(g, *shape, scale=1.0):
    return torch.empty(shape, dtype=BF16, device=DEV).normal_(0, scale, generator=g)


PLACES = (slice(0, 200), slice(524_000, 524_300), slice(WIDE - 300, WIDE))


@pytest.mark.parametrize("T", [3, 300])
def test_widest_output(T):
    """Products whose output is as wide as it may be, and gradients back from it."""
    g = generator(T)
    w, x = normal(g, WIDE, NARROW, scale=1 / 32), normal(g, T, NARROW)
    print("[wide] linear", T, flush=True)
    pre = torch.empty(T, WIDE, dtype=BF16, device=DEV)
    out = B.ep_linear(x, w, act="relu", pre=pre)
    for c in PLACES:
        want, err = P.product64(x.double(), w[c].double().T)
        close(pre[:, c].double(), want, P.rounded(want, err), ("pre", c))
        close(out[:, c].double(), want.clamp_min(0), P.rounded(want, err), ("out", c))
    print("[wide] linear_grad", T, flush=True)
    dx, dw, dbias = B.ep_linear_grad(out, x, w, act="relu", pre=pre)
    for c in PLACES:
        dz = out[:, c].double()                # relu' is 1 where out is not 0
        want, err = P.product64(dz.T, x.double())
        close(dw[c].double(), want, P.rounded(want, err), ("dw", c))
        close(dbias[c].double(), dz.sum(0), (T + 8) * U32 * dz.abs().sum(0), ("dbias", c))
    want = torch.zeros(T, NARROW, dtype=torch.float64, device=DEV)
    size = torch.zeros_like(want)
    for i in range(0, WIDE, 1 << 17):
        d, v = out[:, i:i + (1 << 17)].double(), w[i:i + (1 << 17)].double()
        want += d @ v
        size += d.abs() @ v.abs()
    # the sum of 2^20 terms, whose roundings are of random sign: below 8 sqrt(n) half steps of the size
    close(dx.double(), want, P.rounded(want, 8 * WIDE ** 0.5 * U32 * size), "dx")


@pytest.mark.parametrize("T", [3, 300])
def test_widest_sum(T):
    """A sum of 2^20 - 8 terms, and the gradient of its rows, as wide."""
    g = generator(T + 1)
    w, x = normal(g, NARROW, WIDE, scale=2.0 ** -10), normal(g, T, WIDE)
    print("[wide] linear", T, flush=True)
    out = B.ep_linear(x, w)
    want, size = 0, 0
    for i in range(0, WIDE, 1 << 17):
        v, u = x[:, i:i + (1 << 17)].double(), w[:, i:i + (1 << 17)].double().T
        want = want + v @ u
        size = size + v.abs() @ u.abs()
    close(out.double(), want, P.rounded(want, 8 * WIDE ** 0.5 * U32 * size), "out")
    print("[wide] linear_grad", T, flush=True)
    dx, dw, _ = B.ep_linear_grad(out, x, w)
    for c in PLACES:
        want, err = P.product64(out.double(), w[:, c].double())
        close(dx[:, c].double(), want, P.rounded(want, err), ("dx", c))
        want, err = P.product64(out.double().T, x[:, c].double())
        close(dw[:, c].double(), want, P.rounded(want, err), ("dw", c))


@pytest.mark.parametrize("T", [3, 300])
def test_widest_swiglu(T):
    """SwiGLU of 2I = 2^20 - 16 channels, its gradient with 2I = 2^21 - 16, and fp32 weights' gradients of
    rows as wide."""
    g = generator(T + 2)
    I, n = 2 ** 19 - 8, torch.tensor([T], dtype=torch.int32, device=DEV)
    w13, x = normal(g, 1, 2 * I, NARROW, scale=1 / 32), normal(g, 1, T, NARROW)
    gu = torch.empty(1, T, 2 * I, dtype=BF16, device=DEV)
    print("[wide] swiglu", T, flush=True)
    h = B.ep_expert_swiglu(x, n, w13, T, gu=gu)
    for c in (slice(0, 300), slice(I - 300, I)):
        gate, eg = P.product64(x[0].double(), w13[0, c].double().T)
        up, eu = P.product64(x[0].double(), w13[0, I + c.start:I + c.stop].double().T)
        want, dh = P.swiglu64(gate, up, eg, eu)
        close(h[0][:, c].double(), want, P.rounded(want, dh), ("h", c))
        close(gu[0][:, I + c.start:I + c.stop].double(), up, P.rounded(up, eu), ("up", c))
    del w13, gu, h
    w2, gu = normal(g, 1, NARROW, WIDE, scale=1 / 32), normal(g, 1, T, 2 * WIDE)
    print("[wide] swiglu_dgrad", T, flush=True)
    dgu = B.ep_expert_swiglu_dgrad(x, n, w2, gu, T)
    for c in PLACES:
        dh, err = P.product64(x[0].double(), w2[0][:, c].double())
        gate, up = gu[0][:, c].double(), gu[0][:, WIDE + c.start:WIDE + c.stop].double()
        dg, du, eg, eu = P.swiglu_grad64(dh, err, gate, up)
        close(dgu[0][:, c].double(), dg, P.rounded(dg, eg), ("dg", c))
        close(dgu[0][:, WIDE + c.start:WIDE + c.stop].double(), du, P.rounded(du, eu), ("du", c))
    del w2, dgu
    dy = gu[:, :, :WIDE].contiguous()
    del gu
    for a, b in ((dy, x), (x, dy)):
        dw = torch.full((1, a.shape[2], b.shape[2]), 1.0, device=DEV)
        print("[wide] wgrad", tuple(dw.shape), flush=True)
        B.ep_expert_gemm_wgrad(a, b, n, T, dw=dw, accumulate=True)
        assert all("product_kernel" in k for k in kernels()), kernels()
        for c in PLACES:
            da, db = (a[0][:, c], b[0]) if a is dy else (a[0], b[0][:, c])
            want, err = P.product64(da.double().T, db.double())
            got = dw[0, c] if a is dy else dw[0][:, c]
            close(got.double(), want + 1, err + U32 * ((want + 1).abs() + err), ("dw", c))


def test_most_rows_of_linear_grad():
    """2^21 rows: the most chunks of the bias' sums and the longest weights' gradient."""
    T, H, N = 2 ** 21, 8, 24
    g = generator(5)
    x, w, dout, pre = normal(g, T, H), normal(g, N, H), normal(g, T, N), normal(g, T, N)
    dx, dw, dbias = B.ep_linear_grad(dout, x, w, act="relu", pre=pre)
    dz = dout.double() * (pre > 0)
    # independent roundings, as in a long sum: 8 sqrt(T) half steps of the sum of absolute values
    close(dbias.double(), dz.sum(0), 8 * T ** 0.5 * U32 * dz.abs().sum(0), "dbias")
    want, size = dz.T @ x.double(), dz.T.abs() @ x.double().abs()
    close(dw.double(), want, P.rounded(want, 8 * T ** 0.5 * U32 * size), "dw")
    want, err = P.product64(dz, w.double())
    close(dx.double(), want, P.rounded(want, err), "dx")


# the kernels for few rows, of squares and of tiles
@pytest.mark.parametrize("T", [2, 100, 20000])
def test_subnormal_and_huge_values(T):
    """bf16's subnormal numbers times large ones, and the largest ones times small ones, are exact."""
    H = N = 64
    x = torch.zeros(T, H)
    x[:, 0] = 2.0 ** -130 * (1 + torch.arange(T) % 7)
    x[:, 1] = 255 * 2.0 ** 120
    w = torch.zeros(N, H)
    w[:, 0] = 2.0 ** 100 * (1 + torch.arange(N) % 5)
    w[:, 1] = torch.where(torch.arange(N) % 2 == 0, 0.0, 2.0 ** -126)
    x, w = x.to(BF16), w.to(BF16)
    want, err = P.product64(x.double(), w.double().T)
    close(B.ep_linear(x.to(DEV), w.to(DEV)).cpu().double(), want, P.rounded(want, err), "out")
    wt = w.T.contiguous()                      # dx = dout w with w[k][c]
    dx, dw, _ = B.ep_linear_grad(x.to(DEV), torch.ones(T, H, dtype=BF16, device=DEV), wt.to(DEV))
    close(dx.cpu().double(), want, P.rounded(want, err), "dx")
    want, err = P.product64(x[:, :1].double().T, torch.ones(T, H, dtype=torch.float64))
    close(dw[:1].cpu().double(), want, P.rounded(want, err), "dw")
