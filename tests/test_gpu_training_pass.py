"""A whole MoE block in bf16 forward and backward, from tokens to every gradient, through the public
calls: layout, dispatch, gate/up with SwiGLU, down, combine and a shared expert whose residual is the
combined output. Against the same block in 64 bits; on another stream; captured into a graph."""
import numpy as np
import pytest
import torch

from combine_ep_layout_06_amd import binding as B

pytestmark = pytest.mark.gpu

DEV = "cuda"
BF16 = torch.bfloat16


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    B.load_library()


class Block:
    def __init__(self, T, H, I, E, K, C, S, packed, seed=0):
        self.T, self.H, self.I, self.E, self.K, self.C, self.S = T, H, I, E, K, C, S
        self.packed = packed
        rng = np.random.default_rng(seed)
        r = lambda *s, scale=1.0: torch.from_numpy(  # noqa: E731
            rng.standard_normal(s, dtype=np.float32) * np.float32(scale)).to(BF16)
        self.host = dict(
            x=r(T, H), w13=r(E, 2 * I, H, scale=H ** -0.5), w2=r(E, H, I, scale=I ** -0.5),
            s1=r(S, H, scale=H ** -0.5), b1=r(S), s2=r(H, S, scale=S ** -0.5), b2=r(H),
            dout=r(T, H))
        self.idx = torch.from_numpy(rng.integers(-1, E, size=(T, K)).astype(np.int32))
        self.w = torch.from_numpy(rng.random((T, K), dtype=np.float32))
        self.d = {k: v.to(DEV) for k, v in self.host.items()}
        self.idx_d, self.w_d = self.idx.to(DEV), self.w.to(DEV)
        self.rows = T * K + 15 * E

    def step(self, stream=None):
        """Forward and backward; the outputs and every gradient."""
        d, T, H, I, E, K, C, S = (self.d, self.T, self.H, self.I, self.E, self.K, self.C, self.S)
        kw = dict(stream=stream)
        lead = (self.rows,) if self.packed else (E, C)
        new = lambda *s: B._new(s, BF16, d["x"].device, stream)  # noqa: E731
        recv, gu = new(*lead, H), new(*lead, 2 * I)
        if self.packed:
            lay = B.ep_layout_dispatch_packed(d["x"], self.idx_d, recv, E, C, 1, 16, **kw)
            at = (lay["expert_count"], lay["packed_offset"])
            f = lambda n: getattr(B, n + "_packed")  # noqa: E731
        else:
            lay = B.ep_layout_dispatch(d["x"], self.idx_d, recv, E, C, 1, **kw)
            at = (lay["expert_count"],)
            f = lambda n: getattr(B, n)  # noqa: E731
        pairs = T * K
        h = f("ep_expert_swiglu")(recv, *at, d["w13"], pairs, gu=gu, **kw)
        y = f("ep_expert_gemm")(h, *at, d["w2"], pairs, **kw)
        if self.packed:
            routed = B.ep_combine_packed(y, self.idx_d, lay["slot"], at[1], self.w_d, E, C, **kw)
        else:
            routed = B.ep_combine(y, self.idx_d, lay["slot"], self.w_d, C, **kw)
        pre = new(T, S)
        a = B.ep_linear(d["x"], d["s1"], bias=d["b1"], act="silu", pre=pre, **kw)
        out = B.ep_linear(a, d["s2"], bias=d["b2"], residual=routed, **kw)

        da, ds2, db2 = B.ep_linear_grad(d["dout"], a, d["s2"], **kw)
        dx_shared, ds1, db1 = B.ep_linear_grad(da, d["x"], d["s1"], act="silu", pre=pre, **kw)
        if self.packed:
            dy, dw = B.ep_combine_grad_packed(d["dout"], y, self.idx_d, lay["slot"], at[1], self.w_d,
                                              E, C, **kw)
        else:
            dy, dw = B.ep_combine_grad(d["dout"], y, self.idx_d, lay["slot"], self.w_d, C, **kw)
        dgu = f("ep_expert_swiglu_dgrad")(dy, *at, d["w2"], gu, pairs, **kw)
        dw2 = f("ep_expert_gemm_wgrad")(dy, h, *at, pairs, **kw)
        drecv = f("ep_expert_gemm_dgrad")(dgu, *at, d["w13"], pairs, **kw)
        dw13 = f("ep_expert_gemm_wgrad")(dgu, recv, *at, pairs, **kw)
        ones = self.ones
        if self.packed:
            dx = B.ep_combine_packed(drecv, self.idx_d, lay["slot"], at[1], ones, E, C, **kw)
        else:
            dx = B.ep_combine(drecv, self.idx_d, lay["slot"], ones, C, **kw)
        return dict(out=out, dx=dx, dx_shared=dx_shared, dw=dw, dw13=dw13, dw2=dw2, ds1=ds1, db1=db1,
                    ds2=ds2, db2=db2, slot=lay["slot"])

    @property
    def ones(self):
        if not hasattr(self, "_ones"):
            self._ones = torch.ones(self.T, self.K, device=DEV)
        return self._ones

    def exact(self, slot):
        """The same in 64 bits by autograd on the CPU, without any rounding in between."""
        v = {k: t.double().requires_grad_() for k, t in self.host.items() if k != "dout"}
        w = self.w.double().requires_grad_()
        routed = torch.zeros(self.T, self.H, dtype=torch.float64)
        for e in range(self.E):
            t, j = torch.nonzero((self.idx == e) & (slot >= 0), as_tuple=True)
            g, u = (v["x"][t] @ v["w13"][e].T).chunk(2, 1)
            y = (g * torch.sigmoid(g) * u) @ v["w2"][e].T
            routed = routed.index_add(0, t, w[t, j][:, None] * y)
        z = v["x"] @ v["s1"].T + v["b1"]
        shared = (z * torch.sigmoid(z)) @ v["s2"].T + v["b2"]
        out = routed + shared
        d = self.host["dout"].double()
        gr = torch.autograd.grad(routed, [v["x"], w, v["w13"], v["w2"]], d)
        gs = torch.autograd.grad(shared, [v["x"], v["s1"], v["b1"], v["s2"], v["b2"]], d)
        return dict(out=out.detach(), dx=gr[0], dw=gr[1], dw13=gr[2], dw2=gr[3], dx_shared=gs[0],
                    ds1=gs[1], db1=gs[2], ds2=gs[3], db2=gs[4])


def check(got, want):
    """Every output within 3% of its norm. The chain rounds to bf16 at most six times (x's products, h or
    gu, y, dy, dgu, dx): each a relative error below 2^-8 per element, carried through sums of independent
    terms and factors of order one (silu' u and the like, below 4): 6 * 2^-8 = 2.4%, less on average."""
    for k, v in want.items():
        g = got[k].double().cpu()
        assert torch.isfinite(g).all(), k
        off = float((g - v).norm() / v.norm())
        assert off < 0.03, (k, off)


SHAPES = [(70, 136, 72, 6, 3, 30, 40, False), (70, 136, 72, 6, 3, 30, 40, True),
          (300, 256, 264, 16, 4, 90, 520, False), (513, 264, 136, 5, 2, 300, 136, True)]


@pytest.mark.parametrize("shape", SHAPES)
def test_block_forward_and_backward(shape):
    print(f"[block] {shape}", flush=True)
    b = Block(*shape)
    got = b.step()
    check(got, b.exact(got["slot"].cpu()))


def test_on_another_stream():
    b = Block(*SHAPES[2])
    first = b.step()
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    busy = torch.randn(2048, 2048, device=DEV)
    for _ in range(3):
        for _ in range(20):                    # the current stream stays busy
            busy = torch.tanh(busy @ busy)
        again = b.step(stream=s)
        s.synchronize()
        assert all(torch.equal(first[k], again[k]) for k in first)


def test_two_streams_at_once():
    a, b = Block(*SHAPES[2]), Block(*SHAPES[3])
    fa, fb = a.step(), b.step()
    torch.cuda.synchronize()
    s, t = torch.cuda.Stream(), torch.cuda.Stream()
    for _ in range(3):
        ga, gb = a.step(stream=s), b.step(stream=t)
        s.synchronize()
        t.synchronize()
        assert all(torch.equal(fa[k], ga[k]) for k in fa)
        assert all(torch.equal(fb[k], gb[k]) for k in fb)


@pytest.mark.parametrize("shape", SHAPES[1:3])
def test_captured_into_a_graph(shape):
    """The whole block captured once and replayed on new inputs, with eager work between."""
    b = Block(*shape)
    b.step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = b.step()
    for seed in (1, 2, 3):
        other = Block(*shape, seed=seed)
        for k, v in other.d.items():
            b.d[k].copy_(v)
        b.idx_d.copy_(other.idx_d)
        b.w_d.copy_(other.w_d)
        eager = other.step()
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        kept = {k: v.clone() for k, v in out.items()}
        assert all(torch.equal(kept[k], eager[k]) for k in eager), seed


def test_recorded_calls():
    """record() and replay() of a forward and a backward call."""
    g = torch.Generator(device=DEV)
    g.manual_seed(5)
    x = torch.randn(70, 136, generator=g, device=DEV).to(BF16)
    w = torch.randn(72, 136, generator=g, device=DEV).to(BF16)
    dout = torch.randn(70, 72, generator=g, device=DEV).to(BF16)
    with B.record() as calls:
        out = B.ep_linear(x, w)
        dx, dw, db = B.ep_linear_grad(dout, x, w)
    assert [c[1] for c in calls.calls] == ["ep_linear", "ep_linear_grad"]
    for _ in range(2):
        x.normal_(generator=g)
        calls.replay()
        want = B.ep_linear(x, w), *B.ep_linear_grad(dout, x, w)
        assert all(torch.equal(a, b) for a, b in zip((out, dx, dw, db), want))
