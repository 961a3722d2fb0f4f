"""What the bf16 products, combine's gradient and the dense product refuse, on the CPU: every call below
fails its checks before a kernel could be launched. And the formulas that the GPU tests compare with,
against differences."""
import ctypes

import pytest
import torch

from combine_ep_layout_06_amd import binding as B

import product_reference as P

A16 = 1 << 20          # a fake, 16-byte aligned address: never dereferenced (checks fail first)
INVALID, ALIGN, UNSUPPORTED = B.EP_ERR_INVALID, B.EP_ERR_ALIGN, B.EP_ERR_UNSUPPORTED


@pytest.fixture(scope="module")
def lib():
    return B.load_library()


def shape(T=128, H=2048, E=96, K=8, C=512, R=1):
    return ctypes.byref(B.EpShape(T, H, E, K, C, R))


# entry point, its integers, its pointers in order, which of them need 16-byte alignment, which may be NULL
PRODUCTS = [
    ("ep_expert_gemm", (768,), 4, (0, 2, 3), ()),
    ("ep_expert_swiglu", (768,), 5, (0, 2, 3, 4), (3,)),
    ("ep_expert_gemm_dgrad", (768,), 4, (0, 2, 3), ()),
    ("ep_expert_swiglu_dgrad", (768,), 5, (0, 2, 3, 4), ()),
    ("ep_expert_gemm_wgrad", (768,), 4, (0, 1, 3), ()),
    ("ep_expert_gemm_wgrad_f32", (768, 1), 4, (0, 1, 3), ()),
]
COUNT_AT = {"ep_expert_gemm_wgrad": 2, "ep_expert_gemm_wgrad_f32": 2}


@pytest.mark.parametrize("packed", [False, True])
@pytest.mark.parametrize("name,ints,n,wide,optional", PRODUCTS)
def test_products(lib, name, ints, n, wide, optional, packed):
    fn = getattr(lib, name + ("_packed" if packed else ""))
    count_at = COUNT_AT.get(name, 1)

    def call(sh=None, ints=ints, change=None, rows=1000):
        p = [A16] * n
        if packed:
            p.insert(count_at + 1, A16)
        for k, v in (change or {}).items():
            p[k + (packed and k > count_at)] = v
        lead = (rows, *ints) if packed else ints
        return fn(sh if sh is not None else shape(), *lead, *p, None)

    for kw in (dict(T=-1), dict(H=0), dict(E=0), dict(K=0), dict(C=0), dict(E=96, R=5),
               dict(T=1 << 30), dict(E=1 << 16, C=1 << 16)):
        assert call(shape(**kw)) == INVALID, kw
    assert fn(None, *((1000,) if packed else ()), *ints, *[A16] * (n + packed), None) == INVALID
    assert call(shape(E=2048)) == UNSUPPORTED
    assert call(shape(H=2044)) == UNSUPPORTED
    assert call(shape(H=1 << 20)) == UNSUPPORTED
    assert call(ints=(0, *ints[1:])) == INVALID
    assert call(ints=(-8, *ints[1:])) == INVALID
    assert call(ints=(764, *ints[1:])) == UNSUPPORTED
    assert call(ints=(1 << 20, *ints[1:])) == UNSUPPORTED
    assert call(ints=(524_288, *ints[1:])) == UNSUPPORTED          # 2^30 weights
    assert name in lib.ep_last_error().decode()
    for k in range(n):
        want = 0 if k in optional else INVALID
        if want:
            assert call(change={k: None}) == want, k
        assert call(change={k: A16 + (8 if k in wide else 2)}) == ALIGN, k
    if packed:
        assert call(rows=-1) == INVALID
        p = [A16] * (n + 1)
        p[count_at + 1] = None
        assert fn(shape(), 1000, *ints, *p, None) == INVALID
        p[count_at + 1] = A16 + 2
        assert fn(shape(), 1000, *ints, *p, None) == ALIGN


def test_swiglu_counts_both_halves(lib):
    """2I x H codes below 2^30, and 2I below 2^20."""
    assert lib.ep_expert_swiglu(shape(), 262_144, A16, A16, A16, None, A16, None) == UNSUPPORTED
    assert lib.ep_expert_swiglu(shape(H=8), 1 << 19, A16, A16, A16, None, A16, None) == UNSUPPORTED


def test_combine_grad(lib):
    f, g = lib.ep_combine_grad, lib.ep_combine_grad_packed
    ok = [A16] * 7
    assert f(shape(H=2044), *ok, None) == UNSUPPORTED
    assert f(shape(K=300, E=512), *ok, None) == UNSUPPORTED
    assert f(shape(T=-1), *ok, None) == INVALID
    for k in range(7):
        p = list(ok)
        p[k] = None
        assert f(shape(), *p, None) == INVALID, k
        p[k] = A16 + (8 if k in (0, 1, 5) else 2)
        assert f(shape(), *p, None) == ALIGN, k
    assert g(shape(), -1, *[A16] * 8, None) == INVALID
    assert g(shape(), 10, A16, A16, A16, A16, None, A16, A16, A16, None) == INVALID


def test_linear(lib):
    f, g = lib.ep_linear, lib.ep_linear_grad
    ok = [A16] * 6                     # x, w, bias, residual, pre, out
    for kw, n, act, want in ((dict(T=-1), 768, 0, INVALID), (dict(), 0, 0, INVALID),
                             (dict(), 768, 4, INVALID), (dict(), 768, -1, INVALID),
                             (dict(H=2044), 768, 0, UNSUPPORTED), (dict(), 764, 0, UNSUPPORTED),
                             (dict(), 524_288, 0, UNSUPPORTED), (dict(), 1 << 20, 0, UNSUPPORTED)):
        assert f(shape(**kw), n, act, *ok, None) == want, (kw, n, act)
        assert g(shape(**kw), n, act, *[A16] * 8, 1 << 40, None) == want, (kw, n, act)
    for k in (0, 1, 5):
        assert f(shape(), 768, 0, *[None if i == k else A16 for i in range(6)], None) == INVALID
    for k in range(6):
        assert f(shape(), 768, 0, *[A16 + 8 if i == k else A16 for i in range(6)], None) == ALIGN
    # dout, pre, x, w, dx, dw, dbias, workspace
    need = lib.ep_linear_grad_workspace_bytes(shape(), 768, 2)
    assert need == 768 * (4 * 2 + 2 * 128)
    assert lib.ep_linear_grad_workspace_bytes(shape(), 768, 0) == 768 * 8
    assert lib.ep_linear_grad_workspace_bytes(None, 768, 0) == 0
    assert lib.ep_linear_grad_workspace_bytes(shape(), 768, 9) == 0
    for k in range(8):
        p = [A16] * 8
        p[k] = None
        assert g(shape(), 768, 2, *p, need, None) == INVALID, k
        p[k] = A16 + (2 if k == 6 else 8)
        assert g(shape(), 768, 2, *p, need, None) == ALIGN, k
    assert g(shape(), 768, 2, *[A16] * 8, need - 1, None) == INVALID
    assert "below" in lib.ep_last_error().decode()
    assert g(shape(T=(1 << 21) + 1, K=1), 768, 2, *[A16] * 8, 1 << 40, None) == UNSUPPORTED


def test_binding_refuses_what_does_not_fit():
    E, C, H, N = 3, 5, 16, 24
    z = lambda *s: torch.zeros(s, dtype=torch.bfloat16)  # noqa: E731
    count = torch.zeros(E, dtype=torch.int32)
    offset = torch.zeros(E + 1, dtype=torch.int32)
    x, w, dy, gu = z(E, C, H), z(E, N, H), z(E, C, N), z(E, C, 2 * N)
    bad = [
        lambda: B.ep_expert_gemm(z(E, C, H + 8), count, w, 4),
        lambda: B.ep_expert_gemm(z(E + 1, C, H), count, w, 4),
        lambda: B.ep_expert_gemm(z(C, H), count, w, 4),
        lambda: B.ep_expert_gemm(x, count, z(N, H), 4),
        lambda: B.ep_expert_gemm(x, count, w, 4, y=z(E, C, N + 8)),
        lambda: B.ep_expert_gemm(x, count[:2], w, 4),
        lambda: B.ep_expert_gemm(x.transpose(1, 2).contiguous().transpose(1, 2), count, w, 4),
        lambda: B.ep_expert_gemm_packed(z(9, H), count, count, w, 4),
        lambda: B.ep_expert_gemm_packed(x, count, offset, w, 4),
        lambda: B.ep_expert_swiglu(x, count, z(E, 23, H), 4),
        lambda: B.ep_expert_swiglu(x, count, w, 4, gu=z(E, C, N + 8)),
        lambda: B.ep_expert_gemm_dgrad(x, count, w, 4),
        lambda: B.ep_expert_swiglu_dgrad(x, count, z(E, H, N), dy, 4),
        lambda: B.ep_expert_gemm_wgrad(dy, z(E, C + 1, H), count, 4),
        lambda: B.ep_expert_gemm_wgrad(dy, x, count, 4, dw=z(E, H, N)),
        lambda: B.ep_expert_gemm_wgrad(dy, x, count, 4, accumulate=True),
        lambda: B.ep_combine_grad(z(4, H), x, torch.zeros(4, 2, dtype=torch.int32),
                                  torch.zeros(4, 2, dtype=torch.int32), torch.zeros(4, 2), C + 1),
        lambda: B.ep_linear(z(4, H), z(N, H + 8)),
        lambda: B.ep_linear(z(4, H), z(N, H), act="tanh"),
        lambda: B.linear_grad_workspace_bytes(4, N, "tanh"),
        lambda: B.ep_linear(z(4, H), z(N, H), residual=z(4, N + 8)),
        lambda: B.ep_linear(z(4, H), z(N, H), bias=z(N + 8)),
        lambda: B.ep_linear_grad(z(4, N), z(4, H), z(N, H), act="silu"),
        lambda: B.ep_linear_grad(z(4, N), z(4, H), z(N, H), pre=z(4, N)),
        lambda: B.ep_linear_grad(z(4, N + 8), z(4, H), z(N, H)),
    ]
    for i, f in enumerate(bad):
        with pytest.raises(ValueError):
            f()
            raise AssertionError(i)
    for f in (lambda: B.ep_expert_gemm(x.float(), count, w, 4),
              lambda: B.ep_expert_gemm(x, count.long(), w, 4),
              lambda: B.ep_expert_gemm_wgrad(dy, x, count, 4, dw=z(E, N, H), accumulate=True),
              lambda: B.ep_linear(z(4, H), z(N, H).float()),
              lambda: B.ep_linear_grad(z(4, N), z(4, H), z(N, H), dbias=z(N))):
        with pytest.raises(TypeError):
            f()
    assert gu.shape == (E, C, 2 * N)
    # what fits is refused for its device alone
    with pytest.raises(ValueError, match="current HIP device"):
        B.ep_expert_swiglu(x, count, w, 4)
    with pytest.raises(ValueError, match="current HIP device"):
        B.ep_linear(z(4, H), z(N, H))


def test_formulas_against_differences():
    """The gradients that the GPU results are compared with, against central differences."""
    g = torch.Generator().manual_seed(0)
    z = torch.randn(200, generator=g, dtype=torch.float64) * 3
    z = z[z.abs() > 1e-3]                      # away from relu's corner
    d = 1e-6
    for name in ("none", "relu", "silu", "gelu"):
        diff = (P.act64(name, z + d) - P.act64(name, z - d)) / (2 * d)
        assert (P.act_grad64(name, z) - diff).abs().max() < 1e-8, name
    u = torch.randn(z.shape, generator=g, dtype=torch.float64)
    dh = torch.randn(z.shape, generator=g, dtype=torch.float64)
    h = lambda a, b: P.swiglu64(a, b)[0]  # noqa: E731
    dg, du, _, _ = P.swiglu_grad64(dh, torch.zeros_like(dh), z, u)
    assert (dg - dh * (h(z + d, u) - h(z - d, u)) / (2 * d)).abs().max() < 1e-7
    assert (du - dh * (h(z, u + d) - h(z, u - d)) / (2 * d)).abs().max() < 1e-7


@pytest.mark.parametrize("kw", [dict(E=0, K=0, C=0, R=0), dict(E=-1, K=-1, C=-1, R=-1), dict(E=5, R=2),
                                dict(K=1 << 20), dict(E=1 << 16, C=1 << 16)])
def test_linear_takes_no_part_of_the_shape_but_its_rows(lib, kw):
    """E, K, C and R are not used: whatever they hold, the call gets as far as its next check, and one of
    no rows does nothing."""
    p = [A16 + 8, *[A16] * 5]
    assert lib.ep_linear(shape(T=1 << 20, **kw), 768, 0, *p, None) == ALIGN
    assert lib.ep_linear_grad(shape(T=1 << 20, **kw), 768, 2, A16 + 8, *[A16] * 7, 1 << 40, None) == ALIGN
    assert lib.ep_linear(shape(T=0, **kw), 768, 0, *[A16] * 6, None) == 0


def test_workspace_of_sizes_that_are_refused(lib):
    """0 wherever ep_linear_grad refuses the sizes."""
    f, g = lib.ep_linear_grad_workspace_bytes, lib.ep_linear_grad
    for kw, n, act in ((dict(T=-1), 768, 2), (dict(H=0), 768, 2), (dict(H=-8), 768, 2), (dict(H=2044), 768, 2),
                       (dict(), 764, 2), (dict(), 0, 2), (dict(), -8, 0), (dict(H=1 << 20), 768, 0),
                       (dict(H=8), 1 << 20, 0), (dict(), 524_288, 2), (dict(T=(1 << 21) + 1), 768, 2),
                       (dict(), 768, 4)):
        assert g(shape(**kw), n, act, *[A16] * 8, 1 << 40, None) in (INVALID, UNSUPPORTED), (kw, n)
        assert f(shape(**kw), n, act) == 0, (kw, n, act)
    assert f(shape(T=1 << 21), 520, 3) == 520 * (4 * (1 << 15) + (2 << 21))
    assert f(shape(T=0), 520, 3) == 0


def test_binding_refuses_sizes_beyond_32_bits(lib):
    """A width or a number of rows that the C call would see as its low half (2^32 + 8 as 8)."""
    z = lambda *s, t=torch.bfloat16: torch.empty(s, dtype=t, device="meta")  # noqa: E731
    many, E = 2 ** 32 + 8, 3
    count, offset = z(E, t=torch.int32), z(E + 1, t=torch.int32)
    idx, w = z(4, 2, t=torch.int32), z(4, 2, t=torch.float32)
    for f in (lambda: B.ep_linear(z(4, 8), z(many, 8)),
              lambda: B.ep_linear_grad(z(4, many), z(4, 8), z(many, 8), workspace=z(64)),
              lambda: B.linear_grad_workspace_bytes(4, many, "none"),
              lambda: B.ep_expert_gemm(z(E, 4, 8), count, z(E, many, 8), 4),
              lambda: B.ep_expert_gemm_packed(z(many, 8), count, offset, z(E, 16, 8), 4),
              lambda: B.ep_expert_swiglu(z(E, 4, 8), count, z(E, 2 * many, 8), 4),
              lambda: B.ep_expert_gemm_dgrad(z(E, 4, many), count, z(E, many, 8), 4),
              lambda: B.ep_expert_swiglu_dgrad_packed(z(many, 8), count, offset, z(E, 8, 16), z(many, 32), 4),
              lambda: B.ep_expert_gemm_wgrad_packed(z(many, 16), z(many, 8), count, offset, 4),
              lambda: B.ep_combine_grad_packed(z(4, 8), z(many, 8), idx, idx, offset, w, E, 4)):
        with pytest.raises(ValueError, match="32 bits"):
            f()


def test_grid_of_too_many_threads_is_refused(lib):
    """A launch whose grid has 2^32 threads or more in a dimension, which would wrap, is an error instead:
    combine of 2^27 tokens."""
    s = shape(T=1 << 27, H=8, E=1, K=1, C=1 << 27)
    assert lib.ep_combine(s, *[A16] * 5, None) == B.EP_ERR_HIP
    assert "hipErrorInvalidConfiguration" in lib.ep_last_error().decode()


@pytest.mark.parametrize("name,ints,n,wide,optional", PRODUCTS[:4])
def test_packed_buffers_of_no_rows(lib, name, ints, n, wide, optional):
    """A packed buffer of no rows may be NULL, whatever number of pairs was laid out: nothing to do."""
    p = [A16] * (n + 1)
    for k in range(n):
        if k in wide:
            p[k + (k > 1)] = None
    assert getattr(lib, name + "_packed")(shape(), 0, *ints, *p, None) == 0
    p[2] = None                                # packed_offset
    assert getattr(lib, name + "_packed")(shape(), 0, *ints, *p, None) == INVALID
