"""The experts' bf16 products and their gradients (ep_expert_gemm, ep_expert_swiglu, their dgrad and
wgrad forms, padded and packed) against the definitions in 64 bits: odd row counts, empty experts,
ragged widths, stale and NaN rows that no call may read or write."""
import numpy as np
import pytest
import torch

from combine_ep_layout_06_amd import binding as B

import product_reference as P
from expert_reference import U32

pytestmark = pytest.mark.gpu

DEV = "cuda"
SENTINEL = 0x5A5A


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    B.load_library()


class Experts:
    """E experts' rows in a padded (A = 0) or packed buffer; rows that hold no pair are NaN."""

    def __init__(self, counts, *, C=None, A=0, seed=0):
        self.rng = np.random.default_rng(seed)
        self.counts, self.E, self.packed = counts, len(counts), A > 0
        if self.packed:
            pad = [-(-max(c, 0) // A) * A for c in counts]
            self.first = [int(v) for v in np.cumsum([0] + pad)]
            self.rows = self.first[-1] + 5
            self.C = self.rows
        else:
            self.C = C if C is not None else max([1] + counts)
            self.first = [e * self.C for e in range(self.E + 1)]
            self.rows = self.E * self.C
        self.n = [min(max(c, 0), self.C) for c in counts]
        self.pairs = max(1, sum(self.n))
        self.lead = (self.rows,) if self.packed else (self.E, self.C)
        self.held = torch.zeros(self.rows, dtype=torch.bool)
        for e in range(self.E):
            self.held[self.slice(e)] = True
        self.count = torch.tensor(counts, dtype=torch.int32, device=DEV)
        self.offset = torch.tensor(self.first, dtype=torch.int32, device=DEV)
        self.places = (self.count, self.offset) if self.packed else (self.count,)

    def slice(self, e):
        return slice(self.first[e], self.first[e] + self.n[e])

    def each(self):
        for e in range(self.E):
            if self.n[e]:
                yield e, self.slice(e)

    def random(self, *shape, scale=1.0):
        v = self.rng.standard_normal(shape, dtype=np.float32) * np.float32(scale)
        return torch.from_numpy(v).to(torch.bfloat16)

    def buffer(self, width, scale=1.0):
        b = self.random(self.rows, width, scale=scale)
        b[self.rng.random(b.shape) < 0.01] *= 20
        b[~self.held] = float("nan")
        return b

    def dev(self, b):
        return b.reshape(*self.lead, b.shape[-1]).to(DEV)

    def sentinel(self, width):
        return torch.full((*self.lead, width), SENTINEL, dtype=torch.int16, device=DEV)

    def result(self, out):
        """The rows of an output in 64 bits, after a look at those that hold no pair."""
        out = out.cpu().reshape(self.rows, -1)
        assert (out[~self.held] == SENTINEL).all(), "a row that holds no pair was written"
        return out.view(torch.bfloat16).double()

    def fn(self, name):
        return getattr(B, name + ("_packed" if self.packed else ""))


def close(got, want, tol, what):
    bad = ~((got - want).abs() <= tol)
    assert not bad.any(), (what, int(bad.sum()), float((got - want).abs().max()), float(tol.max()))


def check_forward(x, H, N):
    print(f"[gemm] {x.counts[:8]} E={x.E} H={H} N={N} C={x.C} packed={x.packed}", flush=True)
    rows, w = x.buffer(H), x.random(x.E, N, H, scale=H ** -0.5)
    y = x.sentinel(N)
    x.fn("ep_expert_gemm")(x.dev(rows), *x.places, w.to(DEV), x.pairs, y=y)
    got = x.result(y)
    for e, r in x.each():
        want, err = P.product64(rows[r].double(), w[e].double().T)
        close(got[r], want, P.rounded(want, err), ("gemm", e))
    return y


def check_swiglu(x, H, I, keep):
    print(f"[swiglu] {x.counts[:8]} E={x.E} H={H} I={I} C={x.C} packed={x.packed}", flush=True)
    rows, w = x.buffer(H), x.random(x.E, 2 * I, H, scale=2 * H ** -0.5)
    h, gu = x.sentinel(I), x.sentinel(2 * I) if keep else None
    x.fn("ep_expert_swiglu")(x.dev(rows), *x.places, w.to(DEV), x.pairs, h=h, gu=gu)
    got, kept = x.result(h), x.result(gu) if keep else None
    for e, r in x.each():
        v, err = P.product64(rows[r].double(), w[e].double().T)
        want, dh = P.swiglu64(v[:, :I], v[:, I:], err[:, :I], err[:, I:])
        close(got[r], want, P.rounded(want, dh), ("h", e))
        if keep:
            close(kept[r], v, P.rounded(v, err), ("gu", e))


def check_dgrad(x, H, N):
    print(f"[dgrad] {x.counts[:8]} E={x.E} H={H} N={N} C={x.C} packed={x.packed}", flush=True)
    dy, w = x.buffer(N), x.random(x.E, N, H, scale=N ** -0.5)
    dx = x.sentinel(H)
    x.fn("ep_expert_gemm_dgrad")(x.dev(dy), *x.places, w.to(DEV), x.pairs, dx=dx)
    got = x.result(dx)
    for e, r in x.each():
        want, err = P.product64(dy[r].double(), w[e].double())
        close(got[r], want, P.rounded(want, err), ("dx", e))


def check_swiglu_dgrad(x, H, I, in_place=False):
    print(f"[swiglu_dgrad] {x.counts[:8]} E={x.E} H={H} I={I} C={x.C} packed={x.packed}", flush=True)
    dy, w2, gu = x.buffer(H), x.random(x.E, H, I, scale=H ** -0.5), x.buffer(2 * I)
    gu_d = x.dev(gu)
    if in_place:
        gu_d.view(torch.int16)[~x.held.reshape(x.lead).to(DEV)] = SENTINEL
    dgu = gu_d if in_place else x.sentinel(2 * I)
    x.fn("ep_expert_swiglu_dgrad")(x.dev(dy), *x.places, w2.to(DEV), gu_d, x.pairs, dgu=dgu)
    got = x.result(dgu.view(torch.int16))
    for e, r in x.each():
        dh, err = P.product64(dy[r].double(), w2[e].double())
        g, u = gu[r, :I].double(), gu[r, I:].double()
        dg, du, eg, eu = P.swiglu_grad64(dh, err, g, u)
        close(got[r, :I], dg, P.rounded(dg, eg), ("dg", e))
        close(got[r, I:], du, P.rounded(du, eu), ("du", e))


def check_wgrad(x, H, N, kind="bf16"):
    print(f"[wgrad {kind}] {x.counts[:8]} E={x.E} H={H} N={N} C={x.C} packed={x.packed}", flush=True)
    dy, rows = x.buffer(N), x.buffer(H)
    before = x.random(x.E, N, H).float()
    dw = (torch.full((x.E, N, H), SENTINEL, dtype=torch.int16, device=DEV).view(torch.bfloat16)
          if kind == "bf16" else before.to(DEV) if kind == "accumulate"
          else torch.full((x.E, N, H), float("nan"), device=DEV))
    x.fn("ep_expert_gemm_wgrad")(x.dev(dy), x.dev(rows), *x.places, x.pairs, dw=dw,
                                 accumulate=kind == "accumulate")
    got = dw.cpu().double()
    for e in range(x.E):
        r = x.slice(e)
        want, err = P.product64(dy[r].double().T, rows[r].double())
        if kind == "bf16":
            close(got[e], want, P.rounded(want, err), ("dw", e))
        elif kind == "f32":
            close(got[e], want, err, ("dw", e))
        else:
            b = before[e].double()
            close(got[e], want + b, err + U32 * ((want + b).abs() + err), ("dw", e))


SMALL = [
    # one row, no rows, a full part and one more, a full tile and one more
    dict(counts=[1], A=0), dict(counts=[0, 3, 0], A=0), dict(counts=[64, 65, 0, 63], A=0),
    dict(counts=[256, 257, 255], A=1), dict(counts=[5, 0, 129, 31, 0, 200], A=16),
    dict(counts=[700, 12], A=24),
]
# widths: one chunk, a block's tail, exactly a block and a tile, one chunk more
WIDTHS = [(8, 8), (64, 256), (72, 136), (200, 264), (136, 520), (328, 72)]


@pytest.mark.parametrize("rows", range(len(SMALL)))
@pytest.mark.parametrize("H,N", WIDTHS)
def test_products(rows, H, N):
    x = Experts(**SMALL[rows], seed=rows * 100 + H + N)
    check_forward(x, H, N)
    check_swiglu(x, H, N, keep=True)
    check_dgrad(x, H, N)
    check_swiglu_dgrad(x, H, N)
    for kind in ("bf16", "f32", "accumulate"):
        check_wgrad(x, H, N, kind)
