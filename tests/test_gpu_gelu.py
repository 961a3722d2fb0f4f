"""GELU and its derivative far from 0, against 64 bits: where z Phi(z) is small, an error that is small
beside 1 would be large beside it."""
import pytest
import torch

from combine_ep_layout_06_amd import binding as B

from expert_reference import U16, U32
from test_gpu_products import kernels

pytestmark = pytest.mark.gpu

DEV = "cuda"
BF16 = torch.bfloat16


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    B.load_library()


def phi(z):
    """Phi(z) with its relative accuracy (torch's ndtr takes 1 + erf, which ends at 1e-16)."""
    return torch.special.erfc(-z / 2 ** 0.5) / 2


def share(z):
    """Phi's error bound relative to the smaller tail, as documented."""
    return (1 + z * z) * 2.0 ** -19


# weights of one: z is x exactly. The rows of the kernels for few rows, of the squares and of the tiles
@pytest.mark.parametrize("T,kernel", [(4, "few_rows_kernel"), (300, "square_kernel"), (20000, "product_kernel")])
def test_gelu(T, kernel):
    n = 64
    z = torch.linspace(-13.06, 6, T * n).to(BF16)
    z[: 9] = torch.tensor([-4, -5, -6, -7, -8, -9, -10, -11, -12.0])
    z = z.view(T, n)
    out = B.ep_linear(z.to(DEV), torch.eye(n).to(BF16).to(DEV), act="gelu").cpu().double()
    assert all(kernel in k for k in kernels()), kernels()
    z = z.double()
    want = z * phi(z)
    # z Phi(z): Phi's own error, one rounding of the product, one to bf16
    tail = z.abs() * phi(-z.abs())
    err = tail * share(z) + 3 * U32 * want.abs()
    off = (out - want).abs() - (err + U16 * (want.abs() + err))
    assert off.max() <= 0, (float(off.max()), float(z.flatten()[off.argmax()]))


def test_gelu_grad():
    """dbias of one row is dout * gelu'(pre) in fp32."""
    pre = torch.linspace(-12.5, 12.5, 4096).to(BF16)[None]
    one = torch.ones(1, 8, dtype=BF16, device=DEV)
    dout = torch.ones(1, 4096, dtype=BF16, device=DEV)
    _, _, dbias = B.ep_linear_grad(dout, one, torch.zeros(4096, 8, dtype=BF16, device=DEV), act="gelu",
                                   pre=pre.to(DEV))
    z = pre[0].double()
    tail, bell = phi(-z.abs()), z * torch.exp(-z * z / 2) / (2 * torch.pi) ** 0.5
    want = phi(z) + bell
    # the exponent's argument z^2 / 2 has seven half steps (two for |z| / sqrt(2), twice, and one for its
    # square, two for the change to base 2), the exponential and the factors 8 more. For z > 0
    # Phi is 1 minus its tail, rounded: half a step of fp32 below 1; and the sum is rounded
    err = tail * share(z) + bell.abs() * U32 * (3.5 * z * z + 8) + U32 / 2 * (z > 0) + U32 * want.abs()
    off = (dbias.cpu().double() - want).abs() - err
    assert off.max() <= 0, (float(off.max()), float(z[off.argmax()]))
