"""The whole layer for a few tokens (ep_moe_layer, ep_moe_layer_fp8) against the definition in 64
bits: one token to the most pairs, experts named by none, by all, twice by one token, ids that are
no expert, and its use in graphs, recorded lists and on other streams."""
import numpy as np
import pytest
import torch

from combine_ep_layout_06_amd import binding as B

import expert_reference as R

pytestmark = pytest.mark.gpu

DEV = "cuda"


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    B.load_library()


class Layer:
    def __init__(self, T, E, K, H, I, fp8, idx=None, seed=0):
        print(f"[layer] T={T} E={E} K={K} H={H} I={I} fp8={fp8} seed={seed}", flush=True)
        rng = np.random.default_rng(seed)
        self.T, self.E, self.K, self.H, self.I, self.fp8 = T, E, K, H, I, fp8
        f32 = lambda *s: torch.from_numpy(rng.standard_normal(s, dtype=np.float32))  # noqa: E731
        self.x = f32(T, H).to(torch.bfloat16)
        if idx is None:
            idx = np.argsort(rng.random((T, E)), 1)[:, :K]
        self.idx = torch.from_numpy(np.ascontiguousarray(idx, dtype=np.int32))
        self.w = torch.softmax(f32(T, K), 1)
        if fp8:
            self.w13, self.w2 = R.codes(rng, (E, 2 * I, H), 100), R.codes(rng, (E, H, I), 100)
            scale = lambda n, k: torch.from_numpy(  # noqa: E731
                (np.exp(rng.standard_normal((E, n // 128, k // 128))) / (100 * np.sqrt(k)))
                .astype(np.float32))
            self.s13, self.s2 = scale(2 * I, H), scale(H, I)
        else:
            self.w13 = (f32(E, 2 * I, H) / np.sqrt(H)).to(torch.bfloat16)
            self.w2 = (f32(E, H, I) / np.sqrt(I)).to(torch.bfloat16)
        self.d = {k: getattr(self, k).to(DEV) for k in
                  ("x", "idx", "w", "w13", "w2") + (("s13", "s2") if fp8 else ())}

    def run(self, **kw):
        d = self.d
        if self.fp8:
            return B.ep_moe_layer_fp8(d["x"], d["idx"], d["w"], d["w13"], d["s13"], d["w2"],
                                      d["s2"], **kw)
        return B.ep_moe_layer(d["x"], d["idx"], d["w"], d["w13"], d["w2"], **kw)

    def expected(self):
        held = lambda e: 0 <= e < self.E  # noqa: E731
        if self.fp8:
            return R.layer64(self.x, self.idx, self.w,
                             lambda e: R.weights64(self.w13[e], self.s13[e]) if held(e) else None,
                             lambda e: R.weights64(self.w2[e], self.s2[e]) if held(e) else None)
        return R.layer64(self.x, self.idx, self.w,
                         lambda e: self.w13[e].double() if held(e) else None,
                         lambda e: self.w2[e].double() if held(e) else None)

    def check(self, out=None):
        if out is None:
            ws = torch.full((B.moe_layer_workspace_bytes(self.T, self.K, self.H, self.I) // 4,),
                            float("nan"), device=DEV)
            out = torch.full((self.T, self.H), float("nan"), dtype=torch.bfloat16, device=DEV)
            self.run(out=out, workspace=ws)
            torch.cuda.synchronize()
        want, tol = self.expected()
        bad = (out.cpu().double() - want).abs() > tol
        assert not bad.any() and torch.isfinite(out).all(), (int(bad.sum()), bad.nonzero()[:3])
        return out


SHAPES = [  # T, E, K, H, I
    (1, 1, 1, 128, 128), (1, 8, 2, 256, 128), (1, 128, 8, 512, 256), (3, 5, 5, 384, 128),
    (16, 8, 1, 128, 384), (17, 2, 1, 256, 128), (33, 16, 4, 640, 256), (128, 128, 8, 256, 512),
    (130, 3, 2, 128, 128), (7, 1000, 8, 128, 128), (40, 96, 6, 896, 384),
    # 16 pairs and 17; 16 pairs of one expert; 32 channels of h a workgroup; long rows
    (2, 12, 8, 256, 128), (17, 12, 1, 256, 128), (16, 1, 1, 128, 128), (4, 6, 4, 128, 1024),
    (1, 3, 2, 4096, 256), (2, 2, 2, 128, 2048), (5, 4, 4, 2048, 1152),
]


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("T,E,K,H,I", SHAPES)
def test_layer(T, E, K, H, I, fp8):
    Layer(T, E, K, H, I, fp8, seed=T + E).check()


@pytest.mark.parametrize("T,E,K,H,I", [(1, 4, 2, 64, 64), (5, 7, 3, 192, 64), (20, 4, 2, 320, 448)])
def test_layer_bf16_widths_of_64(T, E, K, H, I):
    Layer(T, E, K, H, I, False, seed=H).check()


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("T,K", [(256, 8), (2048, 1), (8, 256)])
def test_most_pairs(T, K, fp8):
    Layer(T, 256, K, 256, 128, fp8, seed=K).check()


@pytest.mark.parametrize("fp8", [False, True])
def test_one_expert_takes_every_token(fp8):
    idx = np.full((150, 2), 3)
    idx[:, 1] = np.arange(150) % 2                # 150 rows, and 75 each
    Layer(150, 6, 2, 128, 128, fp8, idx=idx, seed=1).check()


@pytest.mark.parametrize("fp8", [False, True])
def test_unrouted_invalid_and_repeated_ids(fp8):
    idx = np.array([[-1, -1, -1], [0, 0, 0], [5, -1, 5], [6, 7, -7], [2 ** 31 - 1, -2 ** 31, 1],
                    [6, 6, 6]])                   # 6 experts: 6 is none
    x = Layer(6, 6, 3, 256, 128, fp8, idx=idx, seed=2)
    out = x.check()
    assert (out[[0, 3, 5]] == 0).all() and not torch.signbit(out[[0, 3, 5]]).any()


@pytest.mark.parametrize("fp8", [False, True])
def test_no_token_names_an_expert(fp8):
    out = Layer(4, 6, 2, 128, 128, fp8, idx=np.full((4, 2), -1), seed=3).check()
    assert (out == 0).all()


def test_no_tokens():
    x = Layer(1, 4, 2, 128, 128, False)
    out = B.ep_moe_layer(x.d["x"][:0], x.d["idx"][:0], x.d["w"][:0], x.d["w13"], x.d["w2"])
    assert out.shape == (0, 128)


@pytest.mark.parametrize("fp8", [False, True])
def test_non_finite_tokens_stay_their_own(fp8):
    """NaN and infinities in one token's row, weight or shared expert reach that token alone."""
    x = Layer(20, 2, 2, 128, 128, fp8, seed=4)
    clean = x.run().cpu()
    x.d["x"][3, 5] = float("nan")
    x.d["x"][7, 6] = float("inf")
    x.d["w"][9, 0] = float("nan")
    out = x.run().cpu()
    hit = torch.zeros(20, dtype=torch.bool)
    hit[[3, 7, 9]] = True
    assert torch.equal(out[~hit], clean[~hit])
    assert torch.isnan(out[3]).all() and torch.isnan(out[9]).all()
    assert not torch.isfinite(out[7]).all()


@pytest.mark.parametrize("fp8", [False, True])
def test_large_values_of_h_keep_their_sign_and_size(fp8):
    """g far below zero gives h = -0, far above gives g * u, up to infinity in out."""
    x = Layer(2, 2, 1, 128, 128, fp8, seed=5)
    x.d["x"].mul_(1e4)
    x.x.mul_(1e4)
    x.check()


@pytest.mark.parametrize("fp8", [False, True])
def test_same_bits_on_another_stream_and_with_another_workspace(fp8):
    x = Layer(24, 16, 4, 256, 256, fp8, seed=6)
    a = x.run()
    torch.cuda.synchronize()
    other = torch.cuda.Stream()
    other.wait_stream(torch.cuda.current_stream())
    ws = torch.empty(B.moe_layer_workspace_bytes(24, 4, 256, 256) + 512, dtype=torch.uint8, device=DEV)
    out = torch.zeros_like(a)
    with torch.cuda.stream(other):
        x.run(out=out, workspace=ws)
    other.synchronize()
    assert torch.equal(a, out)


@pytest.mark.parametrize("fp8", [False, True])
def test_own_workspace_outlives_a_call_on_another_stream(fp8):
    """A workspace allocated by the call is not handed out again while the call's stream is behind."""
    x = Layer(3, 8, 4, 512, 256, fp8, seed=9)
    want = x.run()
    torch.cuda.synchronize()
    other, out = torch.cuda.Stream(), torch.zeros_like(want)
    n = B.moe_layer_workspace_bytes(3, 4, 512, 256)
    torch.cuda.synchronize()
    with torch.cuda.stream(other):
        torch.cuda._sleep(20_000_000)            # about 10 ms
    x.run(out=out, stream=other)
    mine = [torch.zeros(n, dtype=torch.uint8, device=DEV) for _ in range(4)]
    torch.cuda.synchronize()
    assert torch.equal(out, want)
    assert all((m == 0).all() for m in mine), "the layer wrote into memory that was handed out"


@pytest.mark.parametrize("fp8", [False, True])
def test_two_layers_at_once(fp8):
    """Layers on two streams, a workspace each, with nothing between them share no state."""
    xs = [Layer(T, 8, 4, 512, 256, fp8, seed=T) for T in (3, 25)]
    want = [x.run() for x in xs]
    torch.cuda.synchronize()
    ws = [torch.empty(B.moe_layer_workspace_bytes(x.T, 4, 512, 256), dtype=torch.uint8, device=DEV)
          for x in xs]
    out = [torch.zeros_like(w) for w in want]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for _ in range(8):
        for x, o, w, s in zip(xs, out, ws, streams):
            x.run(out=o, workspace=w, stream=s)
    torch.cuda.synchronize()
    for o, w in zip(out, want):
        assert torch.equal(o, w)


@pytest.mark.parametrize("fp8", [False, True])
def test_captured_and_recorded_layers_replay(fp8):
    """A layer captured in a graph and one recorded in a call list, replayed on refilled tokens and
    routes, with eager calls between."""
    x = Layer(9, 12, 3, 256, 128, fp8, seed=7)
    ws = torch.empty(B.moe_layer_workspace_bytes(9, 3, 256, 128), dtype=torch.uint8, device=DEV)
    out, out2 = torch.zeros_like(x.d["x"]), torch.zeros_like(x.d["x"])
    x.run(out=out, workspace=ws)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        x.run(out=out, workspace=ws)
    with B.record() as calls:
        x.run(out=out2, workspace=ws)
    for k in range(3):
        x.d["x"].copy_(torch.randn(9, 256, device=DEV).to(torch.bfloat16))
        x.d["idx"].copy_(torch.randint(-1, 12, (9, 3), device=DEV, dtype=torch.int32))
        g.replay()
        calls.replay()
        torch.cuda.synchronize()
        eager = x.run()
        torch.cuda.synchronize()
        assert torch.equal(out, eager) and torch.equal(out2, eager), k


def test_layer_agrees_with_the_bf16_calls_around_an_expert():
    """One expert per token with weight 1 through dispatch, torch products and combine."""
    x = Layer(30, 5, 1, 256, 128, False, seed=8)
    x.d["w"].fill_(1.0)
    x.w.fill_(1.0)
    out = x.check()
    recv = torch.zeros((5, 30, 256), dtype=torch.bfloat16, device=DEV)
    lay = B.ep_layout_dispatch(x.d["x"], x.d["idx"], recv, 5, 30, 1)
    gu = torch.matmul(recv.float(), x.d["w13"].float().transpose(1, 2))
    h = torch.nn.functional.silu(gu[..., :128]) * gu[..., 128:]
    y = torch.matmul(h, x.d["w2"].float().transpose(1, 2)).to(torch.bfloat16)
    comb = B.ep_combine(y, x.d["idx"], lay["slot"], x.d["w"], 30)
    # the same value but for two different orders of fp32 sums: one step of bf16 apart at most
    step = R.U16 * 2 * comb.float().abs() + 1e-4
    assert ((comb.float() - out.float()).abs() <= step).all()


def diagonal_layer(T, fp8, gate, up, down):
    """A layer of one expert, H = I = 128, whose tokens are ones in the first len(up) channels: gate
    channel c is `gate`, up channel c (-1)^c times the sum of `up`, and W2 `down` on its diagonal.
    Values are (code, power of two), so that FP8 weights hold them exactly too."""
    x = Layer(T, 1, 1, 128, 128, fp8, idx=np.zeros((T, 1)), seed=T)
    x.x.zero_()
    x.x[:, :len(up)] = 1
    x.w.fill_(1.0)
    code = torch.zeros(256, 128, dtype=torch.float64)
    code[:128, 0] = gate[0]
    sign = 1 - 2 * (torch.arange(128) % 2)
    for k, c in enumerate(up):
        code[128:, k] = c[0] * sign
    scale = torch.tensor([gate[1], up[0][1]], dtype=torch.float64)
    code2 = torch.eye(128, dtype=torch.float64) * down[0]
    if fp8:
        f8 = torch.float8_e4m3fn
        x.w13, x.s13 = code.to(f8)[None], scale.float().view(1, 2, 1)
        x.w2, x.s2 = code2.to(f8)[None], torch.full((1, 1, 1), down[1])
    else:
        x.w13 = (code * scale.repeat_interleave(128)[:, None]).to(torch.bfloat16)[None]
        x.w2 = (code2 * down[1]).to(torch.bfloat16)[None]
    for k in x.d:
        x.d[k] = getattr(x, k).to(DEV)
    return x, sign


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("T", [1, 20])
def test_gate_of_minus_88_is_not_lost(T, fp8):
    """1 + exp(88) is above 2^126, its reciprocal subnormal, h of an ordinary size with up = 2^70."""
    x, sign = diagonal_layer(T, fp8, (-88.0, 1.0), [(64.0, 2.0 ** 64)], (1.0, 1.0))
    out = x.run().cpu().double()
    want = -88 / (1 + np.exp(88.0)) * 2.0 ** 70 * sign.double()
    # the exponential's argument (3 |g| + 8 half steps of fp32 for h), h's two parts, out's rounding
    tol = (R.U16 + (3 * 88 + 8) * R.U32 + R.U16 ** 2) * (1 + 2.0 ** -7) * want.abs()
    assert ((out - want).abs() <= tol).all(), (out[0, :2], want[:2])


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("T", [1, 20])
def test_largest_finite_h_stays_finite(T, fp8):
    """h = +-511 * 2^119, finite in fp32 and a tie between the largest bf16 value and infinity: its
    two parts hold it exactly, and out is its product with 2^-100 rounded once (to 2^28)."""
    x, sign = diagonal_layer(T, fp8, (64.0, 2.0 ** 58), [(448.0, 2.0 ** 55), (60.0, 2.0 ** 55),
                                                         (3.0, 2.0 ** 55)], (1.0, 2.0 ** -100))
    out = x.run().cpu().double()
    assert torch.equal(out, (2.0 ** 28 * sign.double()).expand(T, 128)), out[0, :2]


@pytest.mark.parametrize("call", ["layer", "layer_fp8", "layout_ws", "layout_fp8_ws"])
def test_own_workspace_is_memory_of_the_calls_stream(call, monkeypatch):
    """On another stream than torch's current one, a workspace that the call allocates belongs to that
    stream: a block of the current one may have a kernel of its last owner still to come, which the
    call's stream does not wait for. Nothing is launched here."""
    used = []
    empty = torch.empty

    def note(*a, **kw):
        if kw.get("dtype") == torch.uint8:
            used.append(torch.cuda.current_stream())
        return empty(*a, **kw)

    other = torch.cuda.Stream()
    fp8 = call.endswith("fp8") or "fp8" in call
    if call.startswith("layer"):
        x = Layer(3, 8, 4, 512, 256, fp8, seed=9)
        go = lambda out: x.run(out=out, stream=other)  # noqa: E731
        out = torch.zeros_like(x.d["x"])
    else:
        tokens = torch.zeros((8, 128), dtype=torch.bfloat16, device=DEV)
        idx = torch.zeros((8, 2), dtype=torch.int32, device=DEV)
        q, s = torch.zeros((4, 8, 128), dtype=torch.uint8, device=DEV), torch.zeros((4, 8, 1), device=DEV)
        out = torch.zeros((4, 8, 128), dtype=torch.bfloat16, device=DEV)
        go = lambda out: (B.ep_layout_dispatch_fp8_ws(tokens, idx, q, s, 4, 8, 1, stream=other)  # noqa: E731
                          if fp8 else B.ep_layout_dispatch_ws(tokens, idx, out, 4, 8, 1, stream=other))
    monkeypatch.setattr(B, "_call", lambda *a, **kw: None)
    monkeypatch.setattr(torch, "empty", note)
    go(out)
    assert used == [other], used
    assert torch.cuda.current_stream() != other
