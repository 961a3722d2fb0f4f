"""The tiles' kernel where tiles stay whole (more than half as many tiles as workgroups): the dense
product's epilogue and the fp32 weights' gradient on tiles of two, three and four parts of 64 rows."""
import pytest
import torch

from combine_ep_layout_06_amd import binding as B

import product_reference as P
from expert_reference import U32
from test_gpu_gradients import close, linear_inputs, randn, sentinel
from test_gpu_products import Experts, check_wgrad, kernels

pytestmark = pytest.mark.gpu

DEV = "cuda"


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    B.load_library()


# T, H, N with the parts of the tiles that are not cut: 272 tiles for 256 workgroups, all of four (and a
# last round in pieces); 202 of three and two; 135 of four and three; each ends inside a part and inside a
# column tile
TILES = [(4095, 72, 4104), (300, 72, 25608), (700, 200, 11272)]


@pytest.mark.parametrize("T,H,N", TILES)
@pytest.mark.parametrize("act,bias,residual,keep,in_place", [
    ("none", True, True, False, False), ("relu", False, True, True, True),
    ("silu", True, False, True, False), ("gelu", True, True, True, True),
    ("gelu", False, True, False, False)])
def test_linear(T, H, N, act, bias, residual, keep, in_place):
    print(f"[whole tiles] T={T} H={H} N={N} {act} {bias} {residual} {keep} {in_place}", flush=True)
    rng, x, w = linear_inputs(T, H, N)
    b = randn(rng, N) if bias else None
    r = randn(rng, T, N) if residual else None
    out, pre = sentinel(T + 1, N), sentinel(T + 1, N) if keep else None
    if in_place:
        out[:T] = r.to(DEV)
    B.ep_linear(x.to(DEV), w.to(DEV), bias=None if b is None else b.to(DEV), act=act,
                residual=out[:T] if in_place else None if r is None else r.to(DEV),
                pre=pre[:T] if keep else None, out=out[:T])
    assert all("product_kernel" in k for k in kernels()), kernels()
    z, err = P.product64(x.double(), w.double().T)
    if bias:
        z = z + b.double()
        err = err + U32 * (z.abs() + err)
    for buffer in (out, pre) if keep else (out,):
        assert torch.equal(buffer[T:].view(torch.int16), sentinel(1, N).view(torch.int16)), "beyond"
    if keep:
        close(pre[:T].cpu().double(), z, P.rounded(z, err), "pre")
    want = P.act64(act, z)
    # |act'| <= 1.13 for each of them
    err = 1.13 * err + P.act_error(act, z) + 3 * U32 * (want.abs() + 1.13 * err)
    if residual:
        want = want + r.double()
        err = err + U32 * (want.abs() + err)
    close(out[:T].cpu().double(), want, P.rounded(want, err), "out")


# 140 experts' weights: 140 tiles of four parts; 280 of three and two, or of four, 256 of them whole; 420
# of three, all whole in two rounds
@pytest.mark.parametrize("N,H", [(256, 72), (264, 72), (256, 264), (520, 136)])
@pytest.mark.parametrize("kind", ["f32", "accumulate", "bf16"])
def test_wgrad(N, H, kind):
    x = Experts([(e * 37) % 101 for e in range(140)], A=8, seed=N + H)
    check_wgrad(x, H, N, kind)
    assert all("product_kernel" in k for k in kernels()), kernels()
