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


def kernels():
    return [d["kernel"] for d in B.last_launches()]


@pytest.mark.parametrize("mean,E", [(1, 9), (20, 4), (50, 3)])
@pytest.mark.parametrize("A", [0, 8])
def test_few_rows(mean, E, A):
    """The kernel for few rows, with experts that have many more rows than the mean and experts that have
    none; the squares from 33 rows on."""
    counts = [mean] * (E - 2) + [0, 2 * mean]
    x = Experts(counts, A=A, seed=mean)
    for H, N in ((200, 24), (520, 136), (1032, 40)):
        check_forward(x, H, N)
        assert all(("few_rows" if mean <= 32 else "square") + "_kernel" in k for k in kernels()), kernels()
        check_swiglu(x, H, N, keep=True)
        assert all("few_rows_kernel" in k for k in kernels()), kernels()
    check_swiglu(x, 264, 72, keep=False)


def test_few_rows_of_many_experts():
    """Its largest height, where there are more squares than CUs."""
    rng = np.random.default_rng(13)
    x = Experts([int(v) for v in rng.integers(0, 100, 300)], A=8, seed=14)
    check_forward(x, 520, 24)
    assert all("few_rows_kernel" in k for k in kernels()), kernels()


@pytest.mark.parametrize("counts,A", [([300], 0), ([90, 0, 130, 1, 64], 8)])
@pytest.mark.parametrize("H,N", WIDTHS + [(264, 64), (1032, 200), (2056, 8)])
def test_squares(counts, A, H, N):
    """Sums that end inside a step, shorter than the eight wavefronts' steps and longer than a ring."""
    x = Experts(counts, A=A, seed=H + N)
    check_forward(x, H, N)
    assert all("square_kernel" in k for k in kernels()), kernels()


@pytest.mark.parametrize("H,N", [(264, 256), (72, 136), (200, 264), (136, 520), (328, 72)])
def test_forward_of_tiles(H, N):
    rng = np.random.default_rng(H)
    x = Experts([int(v) for v in rng.integers(100, 500, 200)], A=8, seed=H + N)
    check_forward(x, H, N)
    assert all("product_kernel" in k for k in kernels()), kernels()
    check_swiglu(x, H, N, keep=True)
    assert all("product_kernel" in k for k in kernels()), kernels()


@pytest.mark.parametrize("mean,E", [(1, 9), (20, 4), (50, 3)])
@pytest.mark.parametrize("A", [0, 8])
def test_few_rows_dgrad(mean, E, A):
    """The same of the gradient of the rows: sums that end inside a step, shorter than the eight
    wavefronts' steps, as long as a ring of them and much longer; columns that end inside a workgroup's."""
    x = Experts([mean] * (E - 2) + [0, 2 * mean], A=A, seed=mean)
    for H, N in ((8, 8), (72, 24), (200, 264), (136, 1032), (64, 2056)):
        check_dgrad(x, H, N)
        assert all("few_dgrad_kernel" in k for k in kernels()), kernels()
        check_swiglu_dgrad(x, N, H)
        assert all("few_dgrad_kernel" in k for k in kernels()), kernels()
    check_swiglu_dgrad(x, 136, 72, in_place=True)


@pytest.mark.parametrize("H,N", [(8, 8), (264, 256), (72, 136), (200, 264), (136, 520), (328, 72)])
def test_dgrad_of_tiles(H, N):
    rng = np.random.default_rng(H)
    x = Experts([int(v) for v in rng.integers(100, 500, 200)], A=8, seed=H + N)
    check_dgrad(x, H, N)
    assert all("product_kernel" in k for k in kernels()), kernels()
    check_swiglu_dgrad(x, N, H, in_place=H == 200)
    assert all("product_kernel" in k for k in kernels()), kernels()


@pytest.mark.parametrize("pairs", [1, 140, 4096, 10 ** 6])
def test_pairs_do_not_choose_the_rows(pairs):
    """Every row is computed whatever number of pairs the call is told."""
    x = Experts([70, 0, 300, 5], A=0, seed=3)
    x.pairs = pairs
    check_forward(x, 136, 264)
    check_swiglu(x, 136, 72, keep=False)
    check_dgrad(x, 136, 264)
    check_swiglu_dgrad(x, 136, 264)
    check_wgrad(x, 136, 264)


def test_counts_beyond_the_buffers():
    """Counts below 0 and above the capacity, packed offsets outside the buffer."""
    x = Experts([-3, 50, 7], C=20, seed=4)
    for check in (check_forward, check_dgrad, check_swiglu_dgrad, check_wgrad):
        check(x, 72, 136)
    x = Experts([5, 9, 4], A=4, seed=5)
    x.offset[0] = -1                           # no rows
    x.offset[2] = x.rows - 2                   # two of its four
    x.n, x.first = [0, 9, 2], [0, x.first[1], x.rows - 2]
    x.held[:] = False
    for e in range(3):
        x.held[x.slice(e)] = True
    for check in (check_forward, check_dgrad, check_swiglu_dgrad, check_wgrad):
        check(x, 72, 136)


def test_no_rows():
    """No pairs: nothing is written, but the weights' gradient is zero; with pairs and no rows too."""
    x = Experts([0, 0], C=4, seed=6)
    for pairs in (0, 5):
        x.pairs = pairs
        check_forward(x, 64, 72)
        check_swiglu(x, 64, 72, keep=True)
        check_dgrad(x, 64, 72)
        check_swiglu_dgrad(x, 64, 72)
        for kind in ("bf16", "f32", "accumulate"):
            check_wgrad(x, 64, 72, kind)


def test_many_experts():
    """1024 experts, most of them without rows."""
    rng = np.random.default_rng(7)
    counts = [int(v) for v in np.where(rng.random(1024) < 0.1, rng.integers(1, 40, 1024), 0)]
    x = Experts(counts, A=1, seed=8)
    check_forward(x, 72, 40)
    check_dgrad(x, 72, 40)
    check_wgrad(x, 40, 24)


def test_parts_of_tiles():
    """Tiles of one to four parts one after the other in a workgroup's list, over several rounds."""
    rng = np.random.default_rng(9)
    counts = [int(v) for v in rng.integers(0, 700, 120)]
    x = Experts(counts, A=8, seed=10)
    check_forward(x, 72, 776)
    check_swiglu(x, 72, 392, keep=True)
    check_dgrad(x, 776, 72)
    check_swiglu_dgrad(x, 72, 776)
    check_wgrad(x, 264, 520)
    check_wgrad(x, 264, 520, "f32")


def test_same_bits_twice():
    x = Experts([300, 17, 0, 129], A=16, seed=11)
    rows, w = x.dev(x.buffer(264)), x.random(x.E, 520, 264, scale=0.1).to(DEV)
    dy = x.dev(x.buffer(520))
    first = None
    for _ in range(3):
        y, dx = x.sentinel(520), x.sentinel(264)
        B.ep_expert_gemm_packed(rows, *x.places, w, x.pairs, y=y)
        B.ep_expert_gemm_dgrad_packed(dy, *x.places, w, x.pairs, dx=dx)
        dw = B.ep_expert_gemm_wgrad_packed(dy, rows, *x.places, x.pairs).view(torch.int16)
        if first is not None:
            assert all(torch.equal(a, b) for a, b in zip(first, (y, dx, dw)))
        first = (y, dx, dw)


def test_swiglu_gradient_in_place():
    check_swiglu_dgrad(Experts([70, 0, 300, 5], A=8, seed=12), 136, 264, in_place=True)


def test_nan_and_infinity_stay_in_their_rows_and_columns():
    """A NaN or an infinity reaches exactly the elements whose sums it is part of."""
    x = Experts([5, 140], C=140, seed=13)
    H, N = 200, 72
    rows, w = x.buffer(H), x.random(2, N, H, scale=0.1)
    rows[x.slice(1)][7, 3] = float("nan")
    w[1, 9, 199] = float("inf")
    y = x.sentinel(N)
    B.ep_expert_gemm(x.dev(rows), x.count, w.to(DEV), x.pairs, y=y)
    got = x.result(y)
    for e, r in x.each():                      # which elements: on the CPU, row by row
        ref = torch.stack([(rows[i].double() * w[e].double()).sum(1) for i in range(r.start, r.stop)])
        assert torch.equal(torch.isnan(got[r]), torch.isnan(ref))
        assert torch.equal(torch.isinf(got[r]), torch.isinf(ref))
        assert torch.equal(got[r][torch.isinf(ref)], ref[torch.isinf(ref)])
    # gradients: a NaN row of dy reaches its row of dx and every element of dw's columns it enters
    dy = x.buffer(N)
    dy[x.slice(0)][2, 5] = float("nan")
    dx = x.sentinel(H)
    w0 = x.random(2, N, H, scale=0.1)
    B.ep_expert_gemm_dgrad(x.dev(dy), x.count, w0.to(DEV), x.pairs, dx=dx)
    nan = torch.isnan(x.result(dx))[x.held]
    assert nan[2].all() and not nan[torch.arange(len(nan)) != 2].any()
    clean = rows.clone()
    clean[x.slice(1)][7, 3] = 1.0
    dw = torch.isnan(B.ep_expert_gemm_wgrad(x.dev(dy), x.dev(clean), x.count, x.pairs)).cpu()
    assert dw[0, 5].all() and int(dw.sum()) == H


def test_rows_beyond_4_gib():
    """An expert whose rows begin beyond 4 GiB of the buffers, and the others' rows before them."""
    H, N = 4096, 4096
    first = [0, 200, 560_000]
    counts = [130, 7, 90]
    rows = 560_100
    x = torch.empty(rows, H, dtype=torch.bfloat16, device=DEV)
    y = torch.full((rows, N), SENTINEL, dtype=torch.int16, device=DEV)
    g = torch.Generator(device=DEV)
    g.manual_seed(1)
    w = torch.empty(3, N, H, dtype=torch.bfloat16, device=DEV).normal_(0, 1 / 64, generator=g)
    for f, n in zip(first, counts):
        x[f:f + n].normal_(0, 1, generator=g)
    count = torch.tensor(counts, dtype=torch.int32, device=DEV)
    offset = torch.tensor(first + [rows], dtype=torch.int32, device=DEV)
    for fn, out in ((B.ep_expert_gemm_packed, "y"), (B.ep_expert_gemm_dgrad_packed, "dx")):
        y.fill_(SENTINEL)
        print("[beyond 4 GiB]", out, flush=True)
        fn(x, count, offset, w, sum(counts), **{out: y})
        for e, (f, n) in enumerate(zip(first, counts)):
            wide = w[e].double()
            want, err = P.product64(x[f:f + n].double(), wide.T if out == "y" else wide)
            close(y[f:f + n].view(torch.bfloat16).double(), want, P.rounded(want, err), (out, e))
            end = first[e + 1] if e < 2 else rows
            assert (y[f + n:min(end, f + n + 64)] == SENTINEL).all()
    print("[beyond 4 GiB] dw", flush=True)
    dw = B.ep_expert_gemm_wgrad_packed(y.view(torch.bfloat16), x, count, offset, sum(counts))
    for e, (f, n) in enumerate(zip(first, counts)):
        want, err = P.product64(y[f:f + n].view(torch.bfloat16).double().T, x[f:f + n].double())
        close(dw[e].double(), want, P.rounded(want, err), ("dw", e))


def test_more_tiles_than_one_list():
    """More tiles than a workgroup looks up together (64 of 256 workgroups)."""
    T = 64 * 256 * 256 + 3000
    g = torch.Generator(device=DEV)
    g.manual_seed(2)
    x = torch.randn(T, 8, generator=g, device=DEV).to(torch.bfloat16)
    w = torch.randn(8, 8, generator=g, device=DEV).to(torch.bfloat16)
    print("[tiles] linear", T, flush=True)
    out = B.ep_linear(x, w)
    want, err = P.product64(x.double(), w.double().T)
    close(out.double(), want, P.rounded(want, err), "out")
    # weight gradients: 25 tiles for each of 700 experts, three of which have rows
    E, N = 700, 1032
    count = torch.zeros(E, dtype=torch.int32, device=DEV)
    count[3], count[350], count[699] = 5, 70, 1
    dy = torch.randn(E, 70, N, generator=g, device=DEV).to(torch.bfloat16)
    rows = torch.randn(E, 70, N, generator=g, device=DEV).to(torch.bfloat16)
    dw = torch.full((E, N, N), float("nan"), dtype=torch.bfloat16, device=DEV)
    print("[tiles] dw", flush=True)
    B.ep_expert_gemm_wgrad(dy, rows, count, 76, dw=dw)
    held = []
    for e, n in ((3, 5), (350, 70), (699, 1)):
        want, err = P.product64(dy[e, :n].double().T, rows[e, :n].double())
        close(dw[e].double(), want, P.rounded(want, err), ("dw", e))
        held.append(e)
    empty = torch.ones(E, dtype=torch.bool, device=DEV)
    empty[held] = False
    assert (dw[empty] == 0).all()


@pytest.mark.parametrize("counts,A", [([600], 0), ([2000, 0, 1500, 31], 8), ([1, 1600], 24)])
@pytest.mark.parametrize("H,N", [(8, 8), (72, 136), (200, 264), (520, 64)])
def test_wgrad_of_long_sums(counts, A, H, N):
    """Weights' gradients in squares, with sums that end inside a step and experts shorter than the eight
    wavefronts' steps or without rows."""
    x = Experts(counts, A=A, seed=H + N)
    for kind in ("bf16", "f32", "accumulate"):
        check_wgrad(x, H, N, kind)
        assert all("few_wgrad_kernel" in k for k in kernels()), kernels()


def test_wgrad_of_tiles_with_long_sums():
    """Sums as long in the tiles' kernel: more squares than CUs."""
    x = Experts([2000, 0, 1500, 31], A=8, seed=21)
    for kind in ("bf16", "f32", "accumulate"):
        check_wgrad(x, 584, 520, kind)
        assert all("product_kernel" in k for k in kernels()), kernels()


def test_tiles_beyond_2_15():
    """An expert of so many tiles that a tile's number times the parts of 64 rows passes 2^31."""
    T = 12_000_001
    g = torch.Generator(device=DEV)
    g.manual_seed(5)
    x = torch.randn(1, T, 8, generator=g, device=DEV).to(torch.bfloat16)
    w = torch.randn(1, 8, 8, generator=g, device=DEV).to(torch.bfloat16)
    count = torch.tensor([T - 70], dtype=torch.int32, device=DEV)
    for fn, wide in ((B.ep_expert_gemm, w[0].double().T), (B.ep_expert_gemm_dgrad, w[0].double())):
        out = torch.full((1, T, 8), SENTINEL, dtype=torch.int16, device=DEV)
        print("[many tiles]", fn.__name__, flush=True)
        fn(x, count, w, T, **{"y" if fn is B.ep_expert_gemm else "dx": out})
        assert all("product_kernel" in k for k in kernels()), kernels()
        want, err = P.product64(x[0, :T - 70].double(), wide)
        close(out[0, :T - 70].view(torch.bfloat16).double(), want, P.rounded(want, err), fn.__name__)
        assert (out[0, T - 70:] == SENTINEL).all()


def test_long_sum():
    """A weights' gradient over rows whose bytes pass 2^31."""
    T, H, N = 280_000, 4096, 8
    g = torch.Generator(device=DEV)
    g.manual_seed(3)
    x = torch.empty(T, H, dtype=torch.bfloat16, device=DEV).normal_(0, 1, generator=g)
    dy = torch.randn(T, N, generator=g, device=DEV).to(torch.bfloat16)
    dw = torch.zeros(1, N, H, device=DEV)
    count = torch.tensor([T], dtype=torch.int32, device=DEV)
    B.ep_expert_gemm_wgrad(dy[None], x[None], count, T, dw=dw)
    want = torch.zeros(N, H, dtype=torch.float64, device=DEV)
    size = torch.zeros(N, H, dtype=torch.float64, device=DEV)
    for i in range(0, T, 20_000):
        d, v = dy[i:i + 20_000].double(), x[i:i + 20_000].double()
        want += d.T @ v
        size += d.abs().T @ v.abs()
    # the roundings of T additions, each at most half a step of a partial sum, are independent here: a
    # partial sum is below size, and 280000 steps of random sign stay below 8 sqrt(T) half steps of it
    close(dw[0].double(), want, 8 * T ** 0.5 * U32 * size, "dw")


@pytest.mark.parametrize("T", [3, 300])
def test_largest_weights(T):
    """A weight matrix just below 2^30 elements, with the kernel for few rows and with tiles."""
    H, N = 4096, 262_136
    g = torch.Generator(device=DEV)
    g.manual_seed(4)
    w = torch.empty(N, H, dtype=torch.bfloat16, device=DEV).normal_(0, 1 / 64, generator=g)
    x = torch.randn(T, H, generator=g, device=DEV).to(torch.bfloat16)
    out = B.ep_linear(x, w)
    for c in (slice(0, 300), slice(131_000, 131_300), slice(N - 300, N)):
        want, err = P.product64(x.double(), w[c].double().T)
        close(out[:, c].double(), want, P.rounded(want, err), ("out", c))
    dx, dw, _ = B.ep_linear_grad(out, x, w)
    want, err = P.product64(out[:2].double(), w[:, :64].double())
    close(dx[:2, :64].double(), want, P.rounded(want, err), "dx")
    c = slice(N - 300, N)
    want, err = P.product64(out[:, c].double().T, x.double())
    close(dw[c].double(), want, P.rounded(want, err), "dw")


def test_packed_buffers_of_no_rows():
    """Pairs laid out, but a packed buffer of no rows (a tensor without memory): the weights' gradients are
    zero, the rest does nothing. The same of a dense product of no rows."""
    E, H, N = 5, 72, 144
    z = lambda *s: torch.empty(s, dtype=torch.bfloat16, device=DEV)  # noqa: E731
    count = torch.full((E,), 3, dtype=torch.int32, device=DEV)
    offset = torch.zeros(E + 1, dtype=torch.int32, device=DEV)
    at, w = (count, offset), torch.ones(E, N, H, device=DEV).to(torch.bfloat16)
    for pairs in (7, 5000):
        print("[no rows]", pairs, flush=True)
        assert B.ep_expert_gemm_packed(z(0, H), *at, w, pairs).shape == (0, N)
        assert B.ep_expert_swiglu_packed(z(0, H), *at, w, pairs, gu=z(0, N)).shape == (0, N // 2)
        assert B.ep_expert_gemm_dgrad_packed(z(0, N), *at, w, pairs).shape == (0, H)
        assert B.ep_expert_swiglu_dgrad_packed(z(0, N), *at, w, z(0, 2 * H), pairs).shape == (0, 2 * H)
        for kind in ("bf16", "f32", "accumulate"):
            dw = torch.full((E, N, H), 2.0, dtype=torch.bfloat16 if kind == "bf16" else torch.float32,
                            device=DEV)
            B.ep_expert_gemm_wgrad_packed(z(0, N), z(0, H), *at, pairs, dw=dw,
                                          accumulate=kind == "accumulate")
            assert (dw == (2 if kind == "accumulate" else 0)).all(), kind
    idx = torch.zeros(4, 2, dtype=torch.int32, device=DEV)
    dw = torch.full((4, 2), float("nan"), device=DEV)
    B.ep_combine_grad_packed(torch.ones(4, H, device=DEV).to(torch.bfloat16), z(0, H), idx, idx, offset,
                             torch.ones(4, 2, device=DEV), E, 8, dtopk_w=dw)
    assert (dw == 0).all()
    out = B.ep_linear(z(0, H), w[0], bias=w[0, :, 0].contiguous(), act="gelu", pre=z(0, N))
    assert out.shape == (0, N)
    dx, dw, dbias = B.ep_linear_grad(z(0, N), z(0, H), w[0], act="gelu", pre=z(0, N))
    assert dx.shape == (0, H) and (dw == 0).all() and (dbias == 0).all()
