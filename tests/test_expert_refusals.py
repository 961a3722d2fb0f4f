"""Refusals of the experts' operators, on the CPU: the C ABI rejects bad arguments before any
launch, and the Python wrappers reject tensors that do not fit."""
import ctypes

import pytest
import torch

from combine_ep_layout_06_amd import binding as B

A16 = 1 << 20          # a fake aligned address: every call below fails its checks first


@pytest.fixture(scope="module")
def lib():
    return B.load_library()


def shape(T=128, H=2048, E=128, K=8, C=512, R=1):
    return ctypes.byref(B.EpShape(T, H, E, K, C, R))


GEMM = dict(name="ep_expert_gemm_fp8", n=1000, ptrs=6)
SWIGLU = dict(name="ep_expert_swiglu_fp8", n=256, ptrs=7)


def call(lib, op, sh, *, n=None, packed=False, rows=100, at=None, value=None):
    """The call with every pointer aligned but number `at`, which is `value`."""
    args = [A16] * (op["ptrs"] + packed)
    if at is not None:
        args[at] = value
    n = op["n"] if n is None else n
    if packed:
        return getattr(lib, op["name"] + "_packed")(sh, rows, n, *args, None)
    return getattr(lib, op["name"])(sh, n, *args, None)


@pytest.mark.parametrize("packed", [False, True])
@pytest.mark.parametrize("op", [GEMM, SWIGLU], ids=lambda o: o["name"])
def test_product_shapes_refused(lib, op, packed):
    bad = lambda code, sh=None, **kw: call(lib, op, sh or shape(), packed=packed, **kw) == code  # noqa: E731
    assert bad(B.EP_ERR_INVALID, shape(T=-1))
    assert bad(B.EP_ERR_INVALID, shape(H=0))
    assert bad(B.EP_ERR_INVALID, shape(T=1 << 30))
    assert call(lib, op, None, packed=packed) == B.EP_ERR_INVALID
    assert bad(B.EP_ERR_INVALID, n=0) and bad(B.EP_ERR_INVALID, n=-8)
    assert bad(B.EP_ERR_UNSUPPORTED, shape(H=2000))
    assert "multiple of 128" in lib.ep_last_error().decode()
    assert bad(B.EP_ERR_UNSUPPORTED, shape(E=1025))
    assert bad(B.EP_ERR_UNSUPPORTED, n=op["n"] + 4)
    assert bad(B.EP_ERR_UNSUPPORTED, shape(H=1 << 20), n=1024)
    assert "2^30" in lib.ep_last_error().decode()
    assert bad(B.EP_ERR_UNSUPPORTED, shape(H=1 << 24, E=1), n=128)
    if packed:
        assert bad(B.EP_ERR_INVALID, rows=-1)


@pytest.mark.parametrize("packed", [False, True])
@pytest.mark.parametrize("op", [GEMM, SWIGLU], ids=lambda o: o["name"])
def test_product_pointers_refused(lib, op, packed):
    n = op["ptrs"] + packed
    for at in range(n):
        assert call(lib, op, shape(), packed=packed, at=at, value=None) == B.EP_ERR_INVALID, at
        assert call(lib, op, shape(), packed=packed, at=at, value=A16 + 2) == B.EP_ERR_ALIGN, at
    assert lib.ep_last_launches(None, 0) == 0
    # rows, weights and row outputs need 16 bytes; scales, counts and offsets 4
    wide = {0, 3 + packed, 5 + packed}
    for at in wide:
        assert call(lib, op, shape(), packed=packed, at=at, value=A16 + 8) == B.EP_ERR_ALIGN, at


def tensors(E=4, C=8, H=256, N=256):
    return dict(q=torch.zeros((E, C, H), dtype=torch.uint8), s=torch.zeros((E, C, H // 128)),
                count=torch.zeros(E, dtype=torch.int32),
                w=torch.zeros((E, N, H), dtype=torch.uint8),
                ws=torch.zeros((E, -(-N // 128), H // 128)))


@pytest.mark.parametrize("fn", [B.ep_expert_gemm_fp8, B.ep_expert_swiglu_fp8])
@pytest.mark.parametrize("key,value,error", [
    ("q", torch.zeros((4, 8, 256), dtype=torch.int16), TypeError),
    ("q", torch.zeros((4, 8, 512), dtype=torch.uint8), ValueError),
    ("q", torch.zeros((3, 8, 256), dtype=torch.uint8), ValueError),
    ("q", torch.zeros((32, 256), dtype=torch.uint8), ValueError),
    ("q", torch.zeros((4, 256, 8), dtype=torch.uint8).transpose(1, 2), ValueError),
    ("s", torch.zeros((4, 8, 1)), ValueError),
    ("s", torch.zeros((4, 8, 2), dtype=torch.float64), TypeError),
    ("count", torch.zeros(4, dtype=torch.int64), TypeError),
    ("count", torch.zeros(5, dtype=torch.int32), ValueError),
    ("w", torch.zeros((4, 256, 256), dtype=torch.bfloat16), TypeError),
    ("w", torch.zeros((256, 256), dtype=torch.uint8), ValueError),
    ("ws", torch.zeros((4, 1, 2)), ValueError),
])
def test_product_tensors_refused(fn, key, value, error):
    t = tensors()
    t[key] = value
    with pytest.raises(error):
        fn(t["q"], t["s"], t["count"], t["w"], t["ws"], 32)


def test_host_tensors_are_refused():
    t = tensors()
    for fn in (B.ep_expert_gemm_fp8, B.ep_expert_swiglu_fp8):
        with pytest.raises(ValueError, match="current HIP device"):
            fn(t["q"], t["s"], t["count"], t["w"], t["ws"], 32)
    off = torch.zeros(5, dtype=torch.int32)
    for fn in (B.ep_expert_gemm_fp8_packed, B.ep_expert_swiglu_fp8_packed):
        with pytest.raises(ValueError, match="current HIP device"):
            fn(t["q"].view(32, 256), t["s"].view(32, 2), t["count"], off, t["w"], t["ws"], 32)
        with pytest.raises(ValueError):
            fn(t["q"].view(32, 256), t["s"].view(32, 2), t["count"], off[:4], t["w"], t["ws"], 32)
    with pytest.raises(ValueError, match="even"):
        B.ep_expert_swiglu_fp8(t["q"], t["s"], t["count"],
                               torch.zeros((4, 255, 256), dtype=torch.uint8), t["ws"], 32)


# ------------------------------------------------------------------------------------------
# the whole layer
# ------------------------------------------------------------------------------------------

LAYER = dict(T=17, H=256, E=8, K=4, C=1, R=1)


@pytest.mark.parametrize("fp8", [False, True])
def test_layer_shapes_refused(lib, fp8):
    fn, ptrs = (lib.ep_moe_layer_fp8, 8) if fp8 else (lib.ep_moe_layer, 6)
    go = lambda I=128, **kw: fn(shape(**{**LAYER, **kw}), I, *[A16] * (ptrs + 1), 1 << 40, None)  # noqa: E731
    assert go(T=-1) == B.EP_ERR_INVALID and go(I=0) == B.EP_ERR_INVALID
    assert fn(None, 128, *[A16] * (ptrs + 1), 1 << 40, None) == B.EP_ERR_INVALID
    assert go(T=513) == B.EP_ERR_UNSUPPORTED
    assert "EP_MOE_MAX_PAIRS" in lib.ep_last_error().decode()
    assert go(E=1025) == B.EP_ERR_UNSUPPORTED
    assert go(H=320 if fp8 else 288) == B.EP_ERR_UNSUPPORTED
    assert go(I=64 if fp8 else 96) == B.EP_ERR_UNSUPPORTED
    assert go(I=1 << 21) == B.EP_ERR_UNSUPPORTED
    assert go(H=1 << 20, I=256, T=2048, K=1) == B.EP_ERR_UNSUPPORTED
    assert go(T=0) == B.EP_OK and lib.ep_last_launches(None, 0) == 0


@pytest.mark.parametrize("fp8", [False, True])
def test_layer_pointers_refused(lib, fp8):
    fn, ptrs = (lib.ep_moe_layer_fp8, 8) if fp8 else (lib.ep_moe_layer, 6)
    need = 68 * 4 * 128 + 68 * (4 * 256 + 20) + 16          # above 16 pairs: y and the lists too
    assert lib.ep_moe_layer_workspace_bytes(shape(**{**LAYER, "T": 4}), 128) == 16 * 4 * 128
    assert lib.ep_moe_layer_workspace_bytes(shape(**LAYER), 128) == need
    assert lib.ep_moe_layer_workspace_bytes(None, 128) == 0
    assert lib.ep_moe_layer_workspace_bytes(shape(**LAYER), 0) == 0

    def go(at=None, value=None, nbytes=need):
        args = [A16] * (ptrs + 1)
        if at is not None:
            args[at] = value
        return fn(shape(**LAYER), 128, *args, nbytes, None)

    for at in range(ptrs + 1):
        assert go(at, None) == B.EP_ERR_INVALID, at
        assert go(at, A16 + 2) == B.EP_ERR_ALIGN, at
    wide = {0, 3, 5, 7, 8} if fp8 else {0, 3, 4, 5, 6}
    for at in wide:
        assert go(at, A16 + 8) == B.EP_ERR_ALIGN, at
    assert go(nbytes=need - 1) == B.EP_ERR_INVALID
    assert "below" in lib.ep_last_error().decode()


def test_layer_constant_matches_the_header():
    import os
    import re
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    with open(os.path.join(root, "include", "ep.h")) as f:
        assert int(re.search(r"#define EP_MOE_MAX_PAIRS\s+(\d+)", f.read())[1]) == B.EP_MOE_MAX_PAIRS


@pytest.mark.parametrize("change,error", [
    (dict(x=torch.zeros((4, 256))), TypeError),
    (dict(x=torch.zeros((4, 128), dtype=torch.bfloat16)), ValueError),
    (dict(x=torch.zeros((256, 4), dtype=torch.bfloat16).t()), ValueError),
    (dict(idx=torch.zeros((4, 2), dtype=torch.int64)), TypeError),
    (dict(idx=torch.zeros((5, 2), dtype=torch.int32)), ValueError),
    (dict(w=torch.zeros((4, 2), dtype=torch.bfloat16)), TypeError),
    (dict(w13=torch.zeros((3, 128, 256), dtype=torch.bfloat16)), ValueError),
    (dict(w2=torch.zeros((2, 256, 128), dtype=torch.bfloat16)), ValueError),
    (dict(out=torch.zeros((4, 128), dtype=torch.bfloat16)), ValueError),
    (dict(out=torch.zeros((4, 256))), TypeError),
    (dict(workspace=torch.zeros((64, 64)).t()[::2]), ValueError),
    (dict(), ValueError),                                  # host tensors
])
def test_layer_tensors_refused(change, error):
    t = dict(x=torch.zeros((4, 256), dtype=torch.bfloat16), idx=torch.zeros((4, 2), dtype=torch.int32),
             w=torch.zeros((4, 2)), w13=torch.zeros((3, 256, 256), dtype=torch.bfloat16),
             w2=torch.zeros((3, 256, 128), dtype=torch.bfloat16), out=None, workspace=None)
    t.update(change)
    with pytest.raises(error):
        B.ep_moe_layer(t["x"], t["idx"], t["w"], t["w13"], t["w2"], out=t["out"],
                       workspace=t["workspace"])
    if not {"w13", "w2"} & set(change):
        w13, w2 = t["w13"].to(torch.uint8), t["w2"].to(torch.uint8)
        with pytest.raises(error):
            B.ep_moe_layer_fp8(t["x"], t["idx"], t["w"], w13, torch.zeros((3, 2, 2)), w2,
                               torch.zeros((3, 2, 1)), out=t["out"], workspace=t["workspace"])
    if not change:
        with pytest.raises(ValueError, match="w13_scale"):
            B.ep_moe_layer_fp8(t["x"], t["idx"], t["w"], w13, torch.zeros((3, 2, 1)), w2,
                               torch.zeros((3, 2, 1)))


@pytest.mark.parametrize("packed", [False, True])
@pytest.mark.parametrize("op,rows", [(GEMM, 1), (SWIGLU, 2)], ids=["gemm", "swiglu"])
def test_weights_of_2_to_30_codes_are_refused(lib, op, rows, packed):
    """The limit counts an expert's weight rows: N of the product, 2I of the gate and up product.
    With no tokens, a call that passes the checks launches nothing."""
    H = 4096
    at = (1 << 30) // H // rows
    go = lambda n: call(lib, op, shape(T=0, H=H, E=1), n=n, packed=packed)  # noqa: E731
    assert go(at) == B.EP_ERR_UNSUPPORTED and "2^30" in lib.ep_last_error().decode()
    assert go(2 * at - 128) == B.EP_ERR_UNSUPPORTED
    assert go(at - 128) == B.EP_OK and lib.ep_last_launches(None, 0) == 0


def test_layer_workspace_of_shapes_no_call_takes(lib):
    """0 for an invalid shape or size, and no wrapped products of large ones."""
    bytes_of = lambda I=128, **kw: lib.ep_moe_layer_workspace_bytes(shape(**{**LAYER, **kw}), I)  # noqa: E731
    assert bytes_of(T=1 << 30, K=4) == 0                 # T*K above INT32_MAX
    assert bytes_of(E=0) == 0 and bytes_of(T=-1) == 0 and bytes_of(H=0) == 0 and bytes_of(K=0) == 0
    assert bytes_of(I=(1 << 31) - 1, T=(1 << 31) - 1, K=1, H=(1 << 31) - 128) == 0
    assert bytes_of(I=1 << 29, T=(1 << 31) - 1, K=1, H=1 << 29) == ((1 << 31) - 1) * ((8 << 29) + 20) + 16
    assert bytes_of(T=1 << 20, K=1, H=1 << 20, I=1 << 20) == (8 << 40) + (20 << 20) + 16


def test_layer_of_too_many_pairs_allocates_no_workspace(monkeypatch):
    """Such a batch is refused; a workspace for it could be gigabytes."""
    T, K = 4096, 8
    sizes = []
    empty = torch.empty
    monkeypatch.setattr(torch, "empty", lambda *a, **kw: sizes.append(a) or empty(*a, **kw))
    bf16 = lambda *s: torch.zeros(s, dtype=torch.bfloat16)  # noqa: E731
    with pytest.raises((ValueError, RuntimeError)):
        B.ep_moe_layer(bf16(T, 128), torch.zeros((T, K), dtype=torch.int32), torch.zeros((T, K)),
                       bf16(2, 256, 128), bf16(2, 128, 128), out=bf16(T, 128))
    assert all(a[0] <= 4096 for a in sizes), sizes


@pytest.mark.parametrize("pairs", [1 << 32, (1 << 32) + 32, 1 << 31, -(1 << 31) - 1])
def test_pairs_beyond_32_bits_are_refused(pairs):
    """2^32 pairs are not 0 pairs (for which the product would do nothing)."""
    t = tensors()
    with B.record(), pytest.raises(ValueError, match="32 bits"):
        B.ep_expert_gemm_fp8(t["q"], t["s"], t["count"], t["w"], t["ws"], pairs)


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("w2", [(256, 3, 128), (1, 768, 128), (6, 128, 128)])
def test_layer_weights_of_another_order_are_refused(w2, fp8):
    """w2 with as many elements as [E, H, I] and the same I is not [E, H, I]."""
    dtype = torch.uint8 if fp8 else torch.bfloat16
    w13, w2 = torch.zeros((3, 256, 256), dtype=dtype), torch.zeros(w2, dtype=dtype)
    x, idx = torch.zeros((4, 256), dtype=torch.bfloat16), torch.zeros((4, 2), dtype=torch.int32)
    with B.record(), pytest.raises(ValueError, match="do not fit"):
        if fp8:
            B.ep_moe_layer_fp8(x, idx, torch.zeros((4, 2)), w13, torch.zeros((3, 2, 2)), w2,
                               torch.zeros((3, 2, 1)))
        else:
            B.ep_moe_layer(x, idx, torch.zeros((4, 2)), w13, w2)
