"""The experts' FP8 products (ep_expert_gemm_fp8, ep_expert_swiglu_fp8 and their packed forms)
against the definitions in 64 bits: odd row counts, empty experts, ragged widths, stale and NaN
rows that no call may read or write, and the FP8 chain from dispatch to combine."""
import numpy as np
import pytest
import torch

from combine_ep_layout_06_amd import binding as B

import expert_reference as R

pytestmark = pytest.mark.gpu

DEV = "cuda"
NAN8 = 0x7F


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    B.load_library()


class Experts:
    """Rows of E experts in a padded or packed buffer whose other rows hold NaN codes and scales."""

    def __init__(self, counts, H, N, *, C=None, A=0, seed=0, x_scale=1.0):
        rng = np.random.default_rng(seed)
        self.counts, self.H, self.N, self.E = counts, H, N, len(counts)
        self.packed = A > 0
        if self.packed:
            pad = [-(-max(c, 0) // A) * A for c in counts]
            self.first = [int(v) for v in np.cumsum([0] + pad)]
            self.rows = self.first[-1] + 5
            self.C = self.rows
        else:
            self.C = C
            self.first = [e * C for e in range(self.E + 1)]
            self.rows = self.E * C
        self.n = [min(max(c, 0), self.C) for c in counts]
        self.pairs = max(1, sum(self.n))
        self.held = torch.zeros(self.rows, dtype=torch.bool)
        q = torch.full((self.rows, H), NAN8, dtype=torch.uint8)
        s = torch.full((self.rows, H // 128), float("nan"))
        for e in range(self.E):
            r = slice(self.first[e], self.first[e] + self.n[e])
            x = rng.standard_normal((self.n[e], H), dtype=np.float32) * np.float32(x_scale)
            x[rng.random(x.shape) < 0.01] *= 50
            if self.n[e]:
                codes, scale = R.quantise(torch.from_numpy(x))
                q[r], s[r] = codes.view(torch.uint8), scale
            self.held[r] = True
        self.q, self.s = q.view(torch.float8_e4m3fn), s
        self.w_q = R.codes(rng, (self.E, N, H), 100)
        self.w_s = torch.from_numpy(
            (np.exp(rng.standard_normal((self.E, -(-N // 128), H // 128))) / (100 * np.sqrt(H)))
            .astype(np.float32))
        self.offset = torch.tensor(self.first, dtype=torch.int32, device=DEV)
        self.count = torch.tensor(counts, dtype=torch.int32, device=DEV)

    def lead(self):
        return (self.rows,) if self.packed else (self.E, self.C)

    def rows_d(self):
        lead = self.lead()
        return (self.q.reshape(*lead, self.H).to(DEV), self.s.reshape(*lead, -1).to(DEV))

    def each(self):
        for e in range(self.E):
            if self.n[e]:
                yield e, slice(self.first[e], self.first[e] + self.n[e])

    def gemm(self, y, **kw):
        q, s = self.rows_d()
        if self.packed:
            return B.ep_expert_gemm_fp8_packed(q, s, self.count, self.offset, self.w_q.to(DEV),
                                               self.w_s.to(DEV), self.pairs, y=y, **kw)
        return B.ep_expert_gemm_fp8(q, s, self.count, self.w_q.to(DEV), self.w_s.to(DEV),
                                    self.pairs, y=y, **kw)

    def swiglu(self, h_q, h_scale):
        q, s = self.rows_d()
        if self.packed:
            return B.ep_expert_swiglu_fp8_packed(q, s, self.count, self.offset, self.w_q.to(DEV),
                                                 self.w_s.to(DEV), self.pairs, h_q=h_q,
                                                 h_scale=h_scale)
        return B.ep_expert_swiglu_fp8(q, s, self.count, self.w_q.to(DEV), self.w_s.to(DEV),
                                      self.pairs, h_q=h_q, h_scale=h_scale)


def gemm64(x, e, r):
    """The product of rows r of expert e in 64 bits and the bound of its error before rounding."""
    want, err = R.product64(x.q[r], x.s[r], x.w_q[e], x.w_s[e])
    return want, err + R.fp8_product_error(x.q[r], x.s[r], x.w_q[e], x.w_s[e])


def check_gemm(x, pairs=None):
    print(f"[gemm] counts={x.counts} H={x.H} N={x.N} C={x.C} packed={x.packed}", flush=True)
    if pairs is not None:
        x.pairs = pairs
    y = torch.full((*x.lead(), x.N), 0x5A5A, dtype=torch.int16, device=DEV)
    x.gemm(y)
    torch.cuda.synchronize()
    y = y.cpu().reshape(x.rows, x.N)
    assert (y[~x.held] == 0x5A5A).all(), "a row that holds no pair was written"
    v = y.view(torch.bfloat16).double()
    for e, r in x.each():
        want, err = gemm64(x, e, r)
        bad = (v[r] - want).abs() > R.gemm_tolerance(want, err)
        assert not bad.any(), (e, int(bad.sum()), (v[r] - want).abs().max())
    return y


def check_swiglu(x, pairs=None):
    print(f"[swiglu] counts={x.counts} H={x.H} I={x.N // 2} C={x.C} packed={x.packed}", flush=True)
    if pairs is not None:
        x.pairs = pairs
    I = x.N // 2
    h_q = torch.full((*x.lead(), I), 0xA5, dtype=torch.uint8, device=DEV)
    h_s = torch.full((*x.lead(), I // 128), -7.25, device=DEV)
    x.swiglu(h_q, h_s)
    torch.cuda.synchronize()
    h_q, h_s = h_q.cpu().reshape(x.rows, I), h_s.cpu().reshape(x.rows, -1)
    assert (h_q[~x.held] == 0xA5).all() and (h_s[~x.held] == -7.25).all()
    v = h_q.view(torch.float8_e4m3fn).double()
    for e, r in x.each():
        h, dh = R.swiglu64(x.q[r], x.s[r], x.w_q[e], x.w_s[e])
        amax = h.unflatten(1, (-1, 128)).abs().amax(-1)
        damax = dh.unflatten(1, (-1, 128)).amax(-1)
        s = h_s[r].double()
        assert ((s - amax / 448).abs() <= damax / 448 + R.U32 * (amax + damax) / 448).all(), "scale"
        full = s.repeat_interleave(128, 1)
        # a code stands for its value within half a step of E4M3, normal or subnormal (2^-10)
        tol = dh + R.U8 * (h.abs() + dh) * (1 + 2.0 ** -20) + 2.0 ** -10 * full * (1 + 2.0 ** -20)
        bad = (v[r] * full - h).abs() > tol
        assert not bad.any(), (e, int(bad.sum()))
        # the largest code of each block is 448: its scale is its own amax
        top = v[r].abs().unflatten(1, (-1, 128)).amax(-1)
        assert (top[amax > 0] == 448).all()
    return h_q, h_s


PADDED = [
    ([1], 128, 8, 1), ([3], 256, 24, 4), ([0, 1, 0, 2], 128, 136, 2), ([16, 15, 17, 0], 384, 256, 40),
    ([64, 63, 65, 1], 256, 1000, 65), ([130, 0, 127, 128, 129], 640, 264, 130),
    ([-3, 9, 50], 256, 72, 20),               # counts outside [0, C]
    ([300, 20], 1152, 512, 300), ([257], 128, 2048, 257),
]


@pytest.mark.parametrize("counts,H,N,C", PADDED)
def test_gemm_padded(counts, H, N, C):
    check_gemm(Experts(counts, H, N, C=C, seed=len(counts) + H))


@pytest.mark.parametrize("counts,H,N,A", [
    ([1], 128, 8, 1), ([5, 0, 0, 33, 1], 256, 104, 1), ([16, 15, 17], 512, 256, 16),
    ([100, 1, 129, 64], 384, 320, 24), ([200, 0, 131], 128, 520, 128)])
def test_gemm_packed(counts, H, N, A):
    check_gemm(Experts(counts, H, N, A=A, seed=7 + H))


@pytest.mark.parametrize("counts,H,I,C", [
    ([1], 128, 128, 1), ([0, 3, 1], 256, 256, 3), ([16, 15, 17, 0], 384, 128, 40),
    ([65, 0, 130, 127], 256, 384, 130), ([300, 20], 1152, 256, 300)])
def test_swiglu_padded(counts, H, I, C):
    check_swiglu(Experts(counts, H, 2 * I, C=C, seed=H + I))


@pytest.mark.parametrize("counts,H,I,A", [
    ([2], 128, 128, 1), ([5, 0, 0, 33, 1], 256, 128, 1), ([100, 1, 129, 64], 384, 256, 24)])
def test_swiglu_packed(counts, H, I, A):
    check_swiglu(Experts(counts, H, 2 * I, A=A, seed=H + I))


def test_many_experts():
    rng = np.random.default_rng(3)
    counts = [int(c) for c in rng.integers(0, 4, 1024)]
    check_gemm(Experts(counts, 128, 16, C=3, seed=5))
    check_swiglu(Experts(counts, 128, 256, A=1, seed=6))


@pytest.mark.parametrize("pairs", [1, 40, 1000, 100000])
def test_the_number_of_pairs_only_chooses_the_launch(pairs):
    """Any count of pairs computes every row (it sets the tile size and the grid)."""
    check_gemm(Experts([150, 3, 0, 77], 256, 264, C=150, seed=9), pairs=pairs)


@pytest.mark.parametrize("A", [0, 8])
@pytest.mark.parametrize("counts,H", [([256, 128, 1], 128), ([130, 300, 0, 63], 256),
                                      ([256, 129], 2432), ([384], 2048)])
def test_both_tile_heights_give_the_same_bits(counts, H, A):
    """Tiles of 64 and of 128 rows (one workgroup for each tile there is, or 8 workgroups for all,
    which halves the tiles of the busiest): the same sums in the same order."""
    x = Experts(counts, H, 520, C=max(counts), A=A, seed=H)
    a = check_gemm(x)
    assert torch.equal(check_gemm(x, pairs=1), a)
    x = Experts(counts, H, 768, C=max(counts), A=A, seed=H + 1)
    a = check_swiglu(x)
    b = check_swiglu(x, pairs=1)
    assert torch.equal(a[0], b[0]) and torch.equal(a[1].view(torch.int32), b[1].view(torch.int32))


@pytest.mark.parametrize("rows", [1, 70])
def test_a_workgroup_walks_hundreds_of_tiles(rows):
    """8 workgroups for 700 experts of 4 column tiles: more tiles each than it looks up at once."""
    counts = [rows if e % 97 == 0 else e % 2 for e in range(700)]
    counts[3] = 1
    check_gemm(Experts(counts, 128, 776, C=rows, seed=37), pairs=1)
    check_swiglu(Experts(counts, 128, 1024, A=1, seed=38), pairs=1)


def test_rows_beyond_4_gib():
    """The last rows of a packed buffer of 4.5 GB (codes and y): the bits of the same rows in front."""
    x = Experts([3, 5], 2048, 1024, A=1, seed=43)
    rows, n = 2_200_000, 8
    want = torch.zeros((x.rows, 1024), dtype=torch.bfloat16, device=DEV)
    x.gemm(want)
    h_want = [torch.zeros((x.rows, 512), dtype=torch.uint8, device=DEV),
              torch.zeros((x.rows, 4), device=DEV)]
    x.swiglu(*h_want)
    small = x.rows_d()
    q = torch.empty((rows, 2048), dtype=small[0].dtype, device=DEV)
    s = torch.empty((rows, 16), device=DEV)
    q.view(torch.uint8)[-n:], s[-n:] = small[0].view(torch.uint8)[:n], small[1][:n]
    offset = torch.tensor([rows - 8, rows - 5, rows], dtype=torch.int32, device=DEV)
    w_q, w_s = x.w_q.to(DEV), x.w_s.to(DEV)
    y = B.ep_expert_gemm_fp8_packed(q, s, x.count, offset, w_q, w_s, n)
    h_q, h_s = B.ep_expert_swiglu_fp8_packed(q, s, x.count, offset, w_q, w_s, n)
    torch.cuda.synchronize()
    assert torch.equal(y[-n:].view(torch.int16), want[:n].view(torch.int16))
    assert torch.equal(h_q[-n:].view(torch.uint8), h_want[0][:n])
    assert torch.equal(h_s[-n:], h_want[1][:n])


def test_weights_beyond_2_gib():
    """The third expert of three with 2^30 codes each (the most an expert may have)."""
    H, N = 4096, 262144
    gen = torch.Generator(device=DEV).manual_seed(47)
    w = torch.randint(0, 120, (3, N, H), dtype=torch.uint8, device=DEV, generator=gen)
    w_s = torch.rand((3, N // 128, H // 128), device=DEV, generator=gen)
    q = torch.randint(0, 120, (3, 2, H), dtype=torch.uint8, device=DEV, generator=gen)
    s = torch.rand((3, 2, H // 128), device=DEV, generator=gen)
    n = lambda *c: torch.tensor(c, dtype=torch.int32, device=DEV)  # noqa: E731
    with pytest.raises(RuntimeError, match="2\\^30"):
        B.ep_expert_gemm_fp8(q, s, n(0, 0, 2), w, w_s, 2)
    N -= 128                                      # just below
    w, w_s = w.view(-1)[:3 * N * H].view(3, N, H), w_s.view(-1)[:3 * N * H >> 14].view(3, N // 128, -1)
    y = B.ep_expert_gemm_fp8(q, s, n(0, 0, 2), w, w_s, 2)
    alone = B.ep_expert_gemm_fp8(q[2:], s[2:], n(2), w[2:], w_s[2:], 2)
    part = B.ep_expert_gemm_fp8(q[2:], s[2:], n(2), w[2:, -512:], w_s[2:, -4:], 2)
    torch.cuda.synchronize()
    assert torch.equal(y[2].view(torch.int16), alone[0].view(torch.int16))
    assert torch.equal(y[2, :, -512:].view(torch.int16), part[0].view(torch.int16))


def test_two_products_at_once():
    """Calls on two streams with nothing between them share no state."""
    a, b = (Experts([90, 40], 1024, 512, C=90, seed=s) for s in (41, 42))
    ya, yb = (torch.zeros((2, 90, 512), dtype=torch.bfloat16, device=DEV) for _ in range(2))
    held = a.rows_d(), b.rows_d(), a.w_q.to(DEV), b.w_q.to(DEV), a.w_s.to(DEV), b.w_s.to(DEV)
    torch.cuda.synchronize()
    other = torch.cuda.Stream()
    for _ in range(8):
        B.ep_expert_gemm_fp8(*held[0], a.count, held[2], held[4], a.pairs, y=ya)
        B.ep_expert_gemm_fp8(*held[1], b.count, held[3], held[5], b.pairs, y=yb, stream=other)
    torch.cuda.synchronize()
    for x, y in ((a, ya), (b, yb)):
        assert torch.equal(y.cpu().view(torch.int16).reshape(180, 512)[x.held], check_gemm(x)[x.held])


def test_no_pairs_writes_nothing():
    x = Experts([4, 4], 128, 128, C=4)
    x.pairs = 0
    y = torch.full((2, 4, 128), 0x5A5A, dtype=torch.int16, device=DEV)
    x.gemm(y)
    torch.cuda.synchronize()
    assert (y == 0x5A5A).all()


def test_packed_rows_outside_the_buffer_are_left_out():
    """Offsets before, across and past the buffer's end: only rows inside it are written."""
    x = Experts([6, 6, 6, 6], 128, 64, A=8, seed=11)
    x.offset = torch.tensor([-2, 8, x.rows - 3, x.rows + 4, 0], dtype=torch.int32, device=DEV)
    keep = torch.zeros(x.rows, dtype=torch.bool)
    keep[8:14] = True
    keep[x.rows - 3:] = True
    y = torch.full((x.rows, 64), 0x5A5A, dtype=torch.int16, device=DEV)
    x.gemm(y)
    torch.cuda.synchronize()
    y = y.cpu()
    assert (y[~keep] == 0x5A5A).all()
    want, err = gemm64(x, 1, slice(8, 14))
    v = y[8:14].view(torch.bfloat16).double()
    assert ((v - want).abs() <= R.gemm_tolerance(want, err)).all()


@pytest.mark.parametrize("big", [1.0, 16.0, 256.0])
@pytest.mark.parametrize("at,small", [((0, 1), 2), ((0, 15), 7), ((16, 17), 31), ((64, 100), 70)])
def test_matrix_instruction_alignment(big, at, small):
    """The product keeps 13 binary places below the largest exponent of a group of products: with
    +big^2 and -big^2 cancelling, a product 2^-13 of them is still there."""
    x, w = torch.zeros(1, 1, 128), torch.zeros(1, 8, 128)
    x[0, 0, list(at)] = big
    w[0, :, at[0]], w[0, :, at[1]] = big, -big
    x[0, 0, small] = big * 2.0 ** -6
    for c in range(8):
        w[0, c, small] = big * 2.0 ** -c
    f8 = torch.float8_e4m3fn
    y = B.ep_expert_gemm_fp8(x.to(f8).to(DEV), torch.ones(1, 1, 1, device=DEV),
                             torch.ones(1, dtype=torch.int32, device=DEV), w.to(f8).to(DEV),
                             torch.ones(1, 1, 1, device=DEV), 1)
    torch.cuda.synchronize()
    want = (x.double() @ w[0].double().T)[0, 0]
    assert torch.equal(y.cpu().double()[0, 0], want)


def test_non_finite_rows_stay_in_their_own_rows():
    """A NaN code or an infinite scale in one row reaches that row's outputs alone."""
    x = Experts([40, 20], 256, 256, C=40, seed=13)
    q = x.q.view(torch.uint8)
    q[3, 17] = NAN8
    x.s[7, 1] = float("inf")
    y = torch.zeros((2, 40, 256), dtype=torch.bfloat16, device=DEV)
    x.gemm(y)
    h_q = torch.zeros((2, 40, 128), dtype=torch.uint8, device=DEV)
    h_s = torch.zeros((2, 40, 1), device=DEV)
    x.swiglu(h_q, h_s)
    torch.cuda.synchronize()
    y, h_s = y.cpu().reshape(80, 256), h_s.cpu().reshape(80)
    assert torch.isnan(y[3]).all() and not torch.isfinite(y[7]).any()
    assert h_s.view(torch.int32)[3] == 0x7FC00000
    fine = x.held.clone()
    fine[[3, 7]] = False
    assert torch.isfinite(y[fine]).all() and torch.isfinite(h_s[fine]).all()
    assert ((h_q.cpu().reshape(80, 128)[3] & 0x7F) == 0x7F).all()


def test_swiglu_zero_and_tiny_blocks():
    """Rows of zeros give scale 0 and zero codes; blocks whose amax is far below 2^-60 keep the
    cast's rules (the plain encoder)."""
    x = Experts([8], 128, 256, C=8, seed=17)
    x.s[0] = 0.0
    x.s[1] *= 1e-15
    h_q, h_s = check_swiglu_tiny(x)
    assert h_s[0, 0] == 0 and ((h_q[0] & 0x7F) == 0).all()
    assert 0 < h_s[1, 0] < 2.0 ** -60


def check_swiglu_tiny(x):
    h_q = torch.zeros((1, 8, 128), dtype=torch.uint8, device=DEV)
    h_s = torch.zeros((1, 8, 1), device=DEV)
    x.swiglu(h_q, h_s)
    torch.cuda.synchronize()
    h_q, h_s = h_q.cpu()[0], h_s.cpu()[0]
    v = h_q.view(torch.float8_e4m3fn).double() * h_s.double()
    for r in range(1, 8):
        h, dh = R.swiglu64(x.q[r:r + 1], x.s[r:r + 1], x.w_q[0], x.w_s[0])
        tol = dh + R.U8 * (h.abs() + dh) + 2.0 ** -9 * float(h_s[r, 0])
        assert ((v[r] - h[0]).abs() <= tol[0]).all(), r
    return h_q, h_s


def test_same_bits_every_time_and_on_another_stream():
    x = Experts([70, 9, 0, 33], 512, 520, C=70, seed=19)
    a = check_gemm(x)
    y = torch.full((4, 70, 520), 0x5A5A, dtype=torch.int16, device=DEV)
    other = torch.cuda.Stream()
    other.wait_stream(torch.cuda.current_stream())
    x.gemm(y, stream=other)
    other.synchronize()
    assert torch.equal(y.cpu().reshape(280, 520), a)


def test_captured_product_replays():
    """Both products captured into a graph and replayed on refilled rows, with eager work between."""
    x = Experts([20, 3, 0, 50], 256, 512, C=50, seed=23)
    q, s = x.rows_d()
    w_q, w_s = x.w_q.to(DEV), x.w_s.to(DEV)
    d_q, d_s = R.codes(np.random.default_rng(1), (4, 136, 256), 100).to(DEV), torch.rand(4, 2, 2).to(DEV)
    h_q = torch.zeros((4, 50, 256), dtype=torch.uint8, device=DEV)
    h_s = torch.zeros((4, 50, 2), device=DEV)
    y = torch.zeros((4, 50, 136), dtype=torch.bfloat16, device=DEV)

    def step():
        B.ep_expert_swiglu_fp8(q, s, x.count, w_q, w_s, x.pairs, h_q=h_q, h_scale=h_s)
        B.ep_expert_gemm_fp8(h_q, h_s, x.count, d_q, d_s, x.pairs, y=y)

    step()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        step()
    for k in range(3):
        s.mul_(1.5)
        g.replay()
        torch.cuda.synchronize()
        got = y.clone()
        y.zero_()
        step()
        torch.cuda.synchronize()
        assert torch.equal(got, y), k


def test_fp8_chain_from_dispatch_to_combine():
    """Layout + FP8 dispatch, gate/up with SwiGLU, down, combine: against the layer in 64 bits on
    the same quantised rows. The error of each stage is bounded by its own rounding."""
    rng = np.random.default_rng(29)
    T, H, I, E, K, C = 50, 256, 128, 6, 3, 50
    x = torch.from_numpy(rng.standard_normal((T, H), dtype=np.float32)).to(torch.bfloat16)
    idx = torch.from_numpy(np.argsort(rng.random((T, E)), 1)[:, :K].astype(np.int32))
    idx[5] = -1
    w = torch.softmax(torch.from_numpy(rng.standard_normal((T, K)).astype(np.float32)), 1)
    a = Experts([1] * E, H, 2 * I, C=C, seed=31)
    b = Experts([1] * E, I, H, C=C, seed=32)
    q = torch.zeros((E, C, H), dtype=torch.uint8, device=DEV)
    s = torch.zeros((E, C, H // 128), device=DEV)
    lay = B.ep_layout_dispatch_fp8(x.to(DEV), idx.to(DEV), q, s, E, C, 1)
    h_q, h_s = B.ep_expert_swiglu_fp8(q, s, lay["expert_count"], a.w_q.to(DEV), a.w_s.to(DEV), T * K)
    y = B.ep_expert_gemm_fp8(h_q, h_s, lay["expert_count"], b.w_q.to(DEV), b.w_s.to(DEV), T * K)
    out = B.ep_combine(y, idx.to(DEV), lay["slot"], w.to(DEV), C)
    torch.cuda.synchronize()
    slot = lay["slot"].cpu()
    q, s, out = q.cpu().view(torch.float8_e4m3fn), s.cpu(), out.cpu().double()
    for t in range(T):
        want, tol = torch.zeros(H, dtype=torch.float64), torch.zeros(H, dtype=torch.float64)
        for j in range(K):
            e, p = int(idx[t, j]), int(slot[t, j])
            if p < 0:
                continue
            h, dh = R.swiglu64(q[e, p:p + 1], s[e, p:p + 1], a.w_q[e], a.w_s[e])
            # the cast: half a step of E4M3, or of its subnormals (2^-10 of the block's scale)
            dh = dh + R.U8 * (h.abs() + dh) + 2.0 ** -10 * (h.abs() + dh).max() / 448 * 1.01
            w2 = R.weights64(b.w_q[e], b.w_s[e])
            v = (h @ w2.T)[0]
            dv = (dh @ w2.abs().T)[0] + 140 * R.U32 * ((h.abs() + dh) @ w2.abs().T)[0]
            # the FP8 product's cut: 2^-13 of the largest product of each group of 16
            top = lambda m: m.abs().unflatten(1, (-1, 16)).amax(-1)  # noqa: E731
            dv = dv + 16 * 2.0 ** -13 * (top(h.abs() + dh) @ top(w2).T)[0]
            dv = dv + R.U16 * (v.abs() + dv)
            want += w[t, j].double() * v
            tol += w[t, j].double() * (dv + 8 * R.U32 * (v.abs() + dv))
        tol = tol + R.U16 * (want.abs() + tol) + 2.0 ** -133
        assert ((out[t] - want).abs() <= tol).all(), t
    assert (out[5] == 0).all()


def tiles(counts, columns, pairs):
    """(rows of a tile, tiles of the busiest workgroup) by the products' launch and tile rules:
    one workgroup for each tile of 64 rows there can be, up to 256; tiles of 128 rows where they
    leave the busiest less than 5/7 as many; an eighth of the tiles for each eighth of the grid."""
    most_tiles = (pairs // 64 + min(pairs, len(counts))) * columns
    grid = -(-most_tiles // 8) * 8 if most_tiles < 256 else 256
    total = lambda rows: sum(-(-c // rows) for c in counts) * columns  # noqa: E731
    busiest = lambda rows: -(-total(rows) // grid)  # noqa: E731
    rows = 128 if 7 * busiest(128) < 5 * busiest(64) else 64
    return rows, -(-(-(-total(rows) // 8)) // (grid // 8))


@pytest.mark.parametrize("experts,rows,H,height,most", [
    (700, 3, 128, 64, 350),           # a second list of 94 tiles
    (512, 2, 256, 64, 256),           # one full list
    (513, 1, 128, 64, 257),           # a second list of one tile (and, for some workgroups, none)
    (1024, 2, 128, 64, 512),          # two full lists
    (600, 72, 256, 128, 300),         # tall tiles
])
def test_a_workgroup_walks_more_tiles_than_one_list(experts, rows, H, height, most):
    """8 workgroups for every expert's 4 column tiles: the tiles of one are looked up 256 at a time."""
    counts = [max(1, rows - e % 3) for e in range(experts)]
    if rows > 64:
        counts = [rows - e % 5 for e in range(experts)]          # all above one low tile
    assert tiles(counts, 4, 1) == (height, most)
    check_gemm(Experts(counts, H, 776, C=rows, seed=experts), pairs=1)
    check_swiglu(Experts(counts, H, 1024, A=1, seed=experts + 1), pairs=1)


@pytest.mark.parametrize("A", [0, 8])
@pytest.mark.parametrize("counts,columns", [([130, 300, 0, 63], 8), ([0, 129, 0, 0, 255, 1, 192], 4),
                                            ([97, 0, 97], 4)])
def test_both_heights_with_uneven_rests_and_empty_experts(counts, columns, A):
    """The same rows in tiles of 64 rows and of 128, which this asks for: the same bits."""
    pairs = sum(counts)
    assert tiles(counts, columns, pairs)[0] == 64 and tiles(counts, columns, 1)[0] == 128
    x = Experts(counts, 256, 256 * columns - 24, C=max(counts), A=A, seed=columns)
    assert torch.equal(check_gemm(x), check_gemm(x, pairs=1))
    x = Experts(counts, 256, 256 * columns, C=max(counts), A=A, seed=columns + 1)
    a, b = check_swiglu(x), check_swiglu(x, pairs=1)
    assert torch.equal(a[0], b[0]) and torch.equal(a[1].view(torch.int32), b[1].view(torch.int32))


@pytest.mark.parametrize("A", [0, 1])
def test_swiglu_gate_of_minus_88_is_not_lost(A):
    """1 + exp(88) is above 2^126, its reciprocal subnormal, h of an ordinary size where up is large."""
    x = Experts([3], 128, 256, C=3, A=A, seed=53)
    up = torch.arange(1, 128, dtype=torch.uint8)                 # every positive code but NaN
    code = torch.zeros(256, 128, dtype=torch.uint8)
    code[:128, 0] = torch.tensor(-88.0).to(torch.float8_e4m3fn).view(torch.uint8)
    code[128:254, 0] = up[:126]
    code[254:, 0] = up[125]
    x.w_q = code.view(torch.float8_e4m3fn)[None]
    x.w_s = torch.tensor([1.0, 2.0 ** 60]).view(1, 2, 1)
    q = torch.zeros(x.q.shape)
    q[:3, 0] = 1
    x.q, x.s = q.to(torch.float8_e4m3fn), torch.ones(x.s.shape)
    h_q = torch.zeros((*x.lead(), 128), dtype=torch.uint8, device=DEV)
    h_s = torch.zeros((*x.lead(), 1), device=DEV)
    x.swiglu(h_q, h_s)
    h_q, h_s = h_q.cpu().view(x.rows, 128)[:3], h_s.cpu().view(-1)[:3].double()
    want = 88 / (1 + np.exp(88.0)) * 2.0 ** 60                   # times up's code; amax has 448
    assert ((h_s - want).abs() <= (3 * 88 + 8) * R.U32 * want).all(), (h_s, want)
    assert torch.equal(h_q, (code[128:, 0] | 0x80).expand(3, 128))


def test_swiglu_weights_beyond_2_gib():
    """The third expert of three, each with the most codes a gate and up product takes."""
    H, I = 4096, (1 << 17) - 128
    gen = torch.Generator(device=DEV).manual_seed(59)
    w = torch.randint(0, 120, (3, 2 * I, H), dtype=torch.uint8, device=DEV, generator=gen)
    w_s = torch.rand((3, 2 * I // 128, H // 128), device=DEV, generator=gen)
    q = torch.randint(0, 120, (3, 2, H), dtype=torch.uint8, device=DEV, generator=gen)
    s = torch.rand((3, 2, H // 128), device=DEV, generator=gen)
    n = lambda *c: torch.tensor(c, dtype=torch.int32, device=DEV)  # noqa: E731
    h_q, h_s = B.ep_expert_swiglu_fp8(q, s, n(0, 0, 2), w, w_s, 2)
    alone = B.ep_expert_swiglu_fp8(q[2:], s[2:], n(2), w[2:], w_s[2:], 2)
    # the last 256 channels: the last gate rows and the last up rows
    part_w = torch.cat([w[2:, I - 256:I], w[2:, -256:]], 1)
    part_s = torch.cat([w_s[2:, I // 128 - 2:I // 128], w_s[2:, -2:]], 1)
    part = B.ep_expert_swiglu_fp8(q[2:], s[2:], n(2), part_w, part_s, 2)
    torch.cuda.synchronize()
    assert torch.equal(h_q[2], alone[0][0]) and torch.equal(h_s[2], alone[1][0])
    assert torch.equal(h_q[2, :, -256:], part[0][0]) and torch.equal(h_s[2, :, -2:], part[1][0])
    assert torch.isfinite(h_s[2]).all() and (h_s[2] > 0).all()
