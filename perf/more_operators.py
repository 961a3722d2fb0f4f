"""The experts' bf16 operators with their gradients, and the dense product beside them, as measured
cases.

* ``gemm``        the experts' product on bf16 rows: ``y = x @ W[e]^T`` for the rows of each expert.
* ``gemm_bwd``    its gradients: ``dx = dy @ W[e]`` and ``dW[e] = dy^T @ x``, dW in bf16 or fp32.
* ``swiglu``      the gate and up products with ``h = silu(g) * u``; for training ``gu``, the two
                  products in bf16, is kept too.
* ``swiglu_bwd``  from the gradient of the down projection's output: ``dgu`` (through the projection
                  and SwiGLU) and the projection's ``dW``.
* ``combine_grad``  the gradients of the top-k weighted sum: the expert rows' and the weights'.
* ``linear``      a dense product with bias, activation and residual in its epilogue.
* ``linear_bwd``  its gradients: input, weights, bias.

The experts' rows are in the padded receive buffer [E][C] or the packed one [rows]; rows that hold
no pair are left as they were.

With ``own`` false, ``run`` computes them with elementary torch operations in 32 bits; with ``own``
true it calls the library. ``exact`` computes them in 64 bits.
"""
import math

import torch
import torch.nn.functional as F

own = False

BF16 = torch.bfloat16


def listed():
    return [
        # the down projection of the prefill workload (4096 tokens, 96 experts, top-8), capacity
        # 512: the padded receive buffer, every expert's rows end inside a tile
        dict(name="gemm_prefill", op="gemm", packed=False, T=4096, E=96, K=8, H=768, N=2048, C=512,
             A=1, route="uniform"),
        # one token's eight rows on eight of 128 experts: the smallest call, latency and weights
        dict(name="gemm_token", op="gemm", packed=True, T=1, E=128, K=8, H=768, N=2048, C=1, A=1,
             route="uniform"),
        # the down projection's gradients in a training step of 4096 tokens
        dict(name="gemm_bwd_train", op="gemm_bwd", packed=False, T=4096, E=96, K=8, H=768, N=2048,
             C=512, A=1, route="uniform", f32=False),
        # a small, skewed batch in the packed layout, no alignment, odd widths, fp32 gradients
        dict(name="gemm_bwd_ragged", op="gemm_bwd", packed=True, T=777, E=32, K=4, H=1000, N=648,
             C=777, A=1, route="zipf", f32=True),
        # gate and up of a training step: h and what its backward pass needs
        dict(name="swiglu_train", op="swiglu", packed=False, T=4096, E=96, K=8, H=2048, I=768,
             C=512, A=1, route="uniform", keep=True),
        # gate and up of a long prefill on one GPU's 32 large experts: bound by the matrix units
        dict(name="swiglu_large", op="swiglu", packed=True, T=8192, E=32, K=8, H=4096, I=2048,
             C=2560, A=128, route="uniform", keep=False),
        # back through the down projection and SwiGLU in a training step
        dict(name="swiglu_bwd_train", op="swiglu_bwd", packed=False, T=4096, E=96, K=8, H=2048,
             I=768, C=512, A=1, route="uniform"),
        # the combine's gradients of that training step
        dict(name="combine_grad_train", op="combine_grad", packed=False, T=4096, E=96, K=8, H=2048,
             C=512, A=1, route="uniform"),
        # the same for a small batch in the packed layout, routing skewed
        dict(name="combine_grad_small", op="combine_grad", packed=True, T=129, E=128, K=8, H=2056,
             C=129, A=16, route="zipf"),
        # one token through a dense projection with bias and activation: reading the weights
        dict(name="linear_token", op="linear", T=1, H=4096, N=4096, act="gelu", bias=True,
             residual=False, keep=False),
        # the shared expert's second projection on a prefill batch of no round length, added to
        # the routed experts' output
        dict(name="linear_prefill", op="linear", T=4095, H=4096, N=4096, act="none", bias=True,
             residual=True, keep=False),
        # the gradients of a shared expert's first projection in a training step
        dict(name="linear_bwd_train", op="linear_bwd", T=4096, H=2048, N=4096, act="silu"),
    ]


def _log(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(("gemm", "gemm_bwd", "swiglu", "swiglu_bwd", "combine_grad", "linear",
                     "linear_bwd"))
    T = _log(rng, 1, 8192)
    H = 8 * _log(rng, 8, 512)
    if op in ("linear", "linear_bwd"):
        c = dict(op=op, T=T, H=H, N=8 * _log(rng, 8, 1024),
                 act=rng.choice(("none", "relu", "silu", "gelu")))
        if op == "linear":
            c.update(bias=rng.random() < 0.5, residual=rng.random() < 0.5, keep=rng.random() < 0.3)
        return c
    E = _log(rng, 1, 160)
    K = rng.randint(1, min(8, E))
    n = 8 * _log(rng, 8, 512) if op != "combine_grad" else 8
    if op in ("swiglu", "swiglu_bwd"):
        n = 8 * _log(rng, 8, 256)
    while E > K and E * H * n > 96 * 2048 * 1536:
        E = max(K, E // 2)
    C = min(T, int(1.25 * T * K / E) + 16)
    # the plain forms hold E * C rows in 32 bits
    while E * C * (H + 2 * n) > 32 * 2560 * 8192 or E * C * H * n > 16 * 2560 * 4096 * 4096:
        T = max(1, T // 2)
        C = min(T, int(1.25 * T * K / E) + 16)
    packed = rng.random() < 0.5
    c = dict(op=op, packed=packed, T=T, E=E, K=K, H=H, C=C,
             A=rng.choice((1, 16, 24, 128)) if packed else 1,
             route=rng.choice(("uniform", "zipf")))
    if op in ("gemm", "gemm_bwd"):
        c["N"] = n
    if op in ("swiglu", "swiglu_bwd"):
        c["I"] = n
    if op == "gemm_bwd":
        c["f32"] = rng.random() < 0.5
    if op == "swiglu":
        c["keep"] = rng.random() < 0.5
    return c


# ------------------------------------------------------------------------------------------
# inputs
# ------------------------------------------------------------------------------------------

def _route(case, g, dev):
    """K distinct experts for each token, uniformly or by a Zipf(1.2) law over a random order; one
    pair in fifty unrouted."""
    T, E, K = case["T"], case["E"], case["K"]
    keys = -torch.log(-torch.log(torch.rand(T, E, generator=g, device=dev, dtype=torch.float64)))
    if case["route"] == "zipf":
        rank = torch.randperm(E, generator=g, device=dev)
        keys = keys - 1.2 * torch.log(rank + 1.0)
    idx = torch.argsort(keys, dim=1, descending=True)[:, :K].to(torch.int32)
    if case["op"] == "combine_grad":
        idx = torch.where(torch.rand(T, K, generator=g, device=dev) < 0.02, -1, idx)
    return idx.contiguous()


def _layout(case, idx):
    """Slots in token order under the capacity (-1: not kept), counts, and the packed offsets."""
    E, C, A = case["E"], case["C"], case["A"]
    flat = idx.reshape(-1).long()
    seen = F.one_hot(flat + 1, E + 1)[:, 1:]
    place = (seen.cumsum(0) * seen).sum(1) - 1
    slot = torch.where(place < C, place, -1)
    count = seen.sum(0).clamp_max(C)
    padded = (count + A - 1) // A * A
    offset = torch.cat([torch.zeros(1, dtype=torch.long, device=idx.device), padded.cumsum(0)])
    return flat, slot, slot >= 0, count.to(torch.int32), offset.to(torch.int32)


def _rows(n, H, g, dev):
    """bf16 rows, N(0, 1) with one channel value in a hundred 10 times larger."""
    x = torch.randn(n, H, generator=g, device=dev)
    big = torch.rand(n, H, generator=g, device=dev) < 0.01
    return torch.where(big, 10 * x, x).to(BF16)


def _weights(shape, g, dev):
    w = torch.empty(shape, dtype=BF16, device=dev)
    return w.normal_(0, 1 / math.sqrt(shape[-1]), generator=g)


def _prepare_linear(case, g, dev):
    T, H, N = case["T"], case["H"], case["N"]
    s = dict(case=case, x=_rows(T, H, g, dev), w=_weights((N, H), g, dev))
    if case["op"] == "linear":
        s["bias"] = torch.randn(N, generator=g, device=dev).to(BF16) if case["bias"] else None
        s["residual"] = _rows(T, N, g, dev) if case["residual"] else None
        s["out"] = torch.zeros(T, N, dtype=BF16, device=dev)
        s["pre"] = torch.zeros(T, N, dtype=BF16, device=dev) if case["keep"] else None
        return s
    s["dout"] = torch.randn(T, N, generator=g, device=dev).to(BF16)
    s["pre"] = torch.randn(T, N, generator=g, device=dev).to(BF16) if case["act"] != "none" else None
    s["dx"] = torch.zeros(T, H, dtype=BF16, device=dev)
    s["dw"] = torch.zeros(N, H, dtype=BF16, device=dev)
    s["dbias"] = torch.zeros(N, device=dev)
    # a training program keeps one workspace for its largest layer
    s["workspace"] = torch.empty(4 * T * N + 64 * N + (1 << 20), dtype=torch.uint8, device=dev)
    return s


def prepare(case, seed):
    dev = torch.device("cuda", torch.cuda.current_device())
    g = torch.Generator(device=dev)
    g.manual_seed(seed)
    if case["op"] in ("linear", "linear_bwd"):
        return _prepare_linear(case, g, dev)
    T, E, K, H, op = case["T"], case["E"], case["K"], case["H"], case["op"]
    idx = _route(case, g, dev)
    flat, slot, kept, count, offset = _layout(case, idx)
    if case["packed"]:
        rows = min(T * K, E * case["C"]) + E * (case["A"] - 1)
        at = offset[flat].long() + slot
        lead = (rows,)
    else:
        rows = E * case["C"]
        at = flat * case["C"] + slot
        lead = (E, case["C"])
    at = at[kept]
    s = dict(case=case, pairs=T * K, count=count, offset=offset)

    def held(width, values):
        """A receive buffer with `values` in the pairs' rows."""
        b = torch.zeros(rows, width, dtype=BF16, device=dev)
        b[at] = values
        return b.view(*lead, width)

    def buffer(width):
        return torch.zeros(*lead, width, dtype=BF16, device=dev)

    pairs = int(at.numel())
    if op == "combine_grad":
        s.update(idx=idx, slot=slot.to(torch.int32).view(T, K),
                 w=torch.softmax(torch.randn(T, K, generator=g, device=dev), 1),
                 dout=torch.randn(T, H, generator=g, device=dev).to(BF16),
                 y=held(H, _rows(pairs, H, g, dev)), dy=buffer(H),
                 dw=torch.zeros(T, K, device=dev))
        return s
    token = torch.arange(T * K, device=dev)[kept] // K
    x = _rows(T, H, g, dev)[token]
    if op in ("gemm", "gemm_bwd"):
        N = case["N"]
        s.update(x=held(H, x), w=_weights((E, N, H), g, dev))
        if op == "gemm":
            s["y"] = buffer(N)
        else:
            s.update(dy=held(N, torch.randn(pairs, N, generator=g, device=dev).to(BF16)),
                     dx=buffer(H),
                     dw=torch.zeros(E, N, H, dtype=torch.float32 if case["f32"] else BF16,
                                    device=dev))
        return s
    I = case["I"]
    if op == "swiglu":
        s.update(x=held(H, x), w13=_weights((E, 2 * I, H), g, dev), h=buffer(I),
                 gu=buffer(2 * I) if case["keep"] else None)
    else:
        gu = torch.randn(pairs, 2 * I, generator=g, device=dev).to(BF16)
        gate, up = gu.float().chunk(2, 1)
        h = (gate / (1 + torch.exp(-gate)) * up).to(BF16)
        s.update(dy=held(H, torch.randn(pairs, H, generator=g, device=dev).to(BF16)),
                 w2=_weights((E, H, I), g, dev), gu=held(2 * I, gu), h=held(I, h),
                 dgu=buffer(2 * I), dw2=torch.zeros(E, H, I, dtype=BF16, device=dev))
    return s


# ------------------------------------------------------------------------------------------
# the operators
# ------------------------------------------------------------------------------------------

def run(state):
    name = state["case"]["op"]
    return globals()[("_own_" if own else "_plain_") + name](state)


def _own_gemm(s):
    from combine_ep_layout_06_amd import binding as B
    if s["case"]["packed"]:
        return B.ep_expert_gemm_packed(s["x"], s["count"], s["offset"], s["w"], s["pairs"],
                                       y=s["y"])
    return B.ep_expert_gemm(s["x"], s["count"], s["w"], s["pairs"], y=s["y"])


def _own_gemm_bwd(s):
    from combine_ep_layout_06_amd import binding as B
    if s["case"]["packed"]:
        dx = B.ep_expert_gemm_dgrad_packed(s["dy"], s["count"], s["offset"], s["w"], s["pairs"],
                                           dx=s["dx"])
        dw = B.ep_expert_gemm_wgrad_packed(s["dy"], s["x"], s["count"], s["offset"], s["pairs"],
                                           dw=s["dw"])
    else:
        dx = B.ep_expert_gemm_dgrad(s["dy"], s["count"], s["w"], s["pairs"], dx=s["dx"])
        dw = B.ep_expert_gemm_wgrad(s["dy"], s["x"], s["count"], s["pairs"], dw=s["dw"])
    return dx, dw


def _own_swiglu(s):
    from combine_ep_layout_06_amd import binding as B
    if s["case"]["packed"]:
        h = B.ep_expert_swiglu_packed(s["x"], s["count"], s["offset"], s["w13"], s["pairs"],
                                      h=s["h"], gu=s["gu"])
    else:
        h = B.ep_expert_swiglu(s["x"], s["count"], s["w13"], s["pairs"], h=s["h"], gu=s["gu"])
    return (h, s["gu"]) if s["case"]["keep"] else h


def _own_swiglu_bwd(s):
    from combine_ep_layout_06_amd import binding as B
    if s["case"]["packed"]:
        dgu = B.ep_expert_swiglu_dgrad_packed(s["dy"], s["count"], s["offset"], s["w2"], s["gu"],
                                              s["pairs"], dgu=s["dgu"])
        dw2 = B.ep_expert_gemm_wgrad_packed(s["dy"], s["h"], s["count"], s["offset"], s["pairs"],
                                            dw=s["dw2"])
    else:
        dgu = B.ep_expert_swiglu_dgrad(s["dy"], s["count"], s["w2"], s["gu"], s["pairs"],
                                       dgu=s["dgu"])
        dw2 = B.ep_expert_gemm_wgrad(s["dy"], s["h"], s["count"], s["pairs"], dw=s["dw2"])
    return dgu, dw2


def _own_combine_grad(s):
    from combine_ep_layout_06_amd import binding as B
    c = s["case"]
    if c["packed"]:
        return B.ep_combine_grad_packed(s["dout"], s["y"], s["idx"], s["slot"], s["offset"],
                                        s["w"], c["E"], c["C"], dy=s["dy"], dtopk_w=s["dw"])
    return B.ep_combine_grad(s["dout"], s["y"], s["idx"], s["slot"], s["w"], c["C"], dy=s["dy"],
                             dtopk_w=s["dw"])


def _own_linear(s):
    from combine_ep_layout_06_amd import binding as B
    c = s["case"]
    out = B.ep_linear(s["x"], s["w"], bias=s["bias"], act=c["act"], residual=s["residual"],
                      pre=s["pre"], out=s["out"])
    return (out, s["pre"]) if c["keep"] else out


def _own_linear_bwd(s):
    from combine_ep_layout_06_amd import binding as B
    return B.ep_linear_grad(s["dout"], s["x"], s["w"], act=s["case"]["act"], pre=s["pre"],
                            dx=s["dx"], dw=s["dw"], dbias=s["dbias"], workspace=s["workspace"])


def _grid(s, v):
    """The pairs' rows of a buffer as [E, C, n] in 32 bits, zeros where there is none."""
    c = s["case"]
    held = torch.arange(c["C"], device=v.device) < s["count"][:, None]
    if c["packed"]:
        at = s["offset"][:-1, None].long() + torch.arange(c["C"], device=v.device)
        v = v[at.clamp_max(v.shape[0] - 1)]
    return torch.where(held[..., None], v.float(), 0.0)


def _place(s, v, before):
    """v [E, C, n] where a pair's row is, `before` elsewhere."""
    c = s["case"]
    v = v.to(before.dtype)
    if not c["packed"]:
        held = torch.arange(c["C"], device=v.device) < s["count"][:, None]
        return torch.where(held[..., None], v, before)
    row = torch.arange(before.shape[0], device=v.device, dtype=torch.int32)
    e = torch.searchsorted(s["offset"][1:], row, right=True).clamp_max(c["E"] - 1)
    slot = row - s["offset"][e]
    held = slot < s["count"][e]
    return torch.where(held[:, None], v[e, slot.clamp(0, c["C"] - 1).long()], before)


def _plain_gemm(s):
    return _place(s, torch.matmul(_grid(s, s["x"]), s["w"].float().transpose(1, 2)), s["y"])


def _plain_gemm_bwd(s):
    dy, x = _grid(s, s["dy"]), _grid(s, s["x"])
    dx = _place(s, torch.matmul(dy, s["w"].float()), s["dx"])
    return dx, torch.matmul(dy.transpose(1, 2), x).to(s["dw"].dtype)


def _plain_swiglu(s):
    v = torch.matmul(_grid(s, s["x"]), s["w13"].float().transpose(1, 2))
    gate, up = v.chunk(2, -1)
    h = _place(s, gate / (1 + torch.exp(-gate)) * up, s["h"])
    return (h, _place(s, v, s["gu"])) if s["case"]["keep"] else h


def _plain_swiglu_bwd(s):
    dy = _grid(s, s["dy"])
    dh = torch.matmul(dy, s["w2"].float())
    gate, up = _grid(s, s["gu"]).chunk(2, -1)
    sig = 1 / (1 + torch.exp(-gate))
    dgu = torch.cat([dh * up * sig * (1 + gate * (1 - sig)), dh * gate * sig], -1)
    dw2 = torch.matmul(dy.transpose(1, 2), _grid(s, s["h"])).to(s["dw2"].dtype)
    return _place(s, dgu, s["dgu"]), dw2


def _plain_combine_grad(s):
    c = s["case"]
    T, K = c["T"], c["K"]
    kept = s["slot"] >= 0
    e = s["idx"].long().clamp_min(0)
    base = s["offset"].long()[e] if c["packed"] else e * c["C"]
    at = torch.where(kept, base + s["slot"], 0)
    dout = s["dout"].float()
    y = s["y"].view(-1, c["H"])[at].float()
    dw = torch.where(kept, (y * dout[:, None]).sum(-1), 0.0)
    # where each row's pair is: one past the last pair for a row that holds none
    rows = s["y"].numel() // c["H"]
    pair = torch.full((rows + 1,), T * K, device=y.device)
    pair[torch.where(kept, at, rows).reshape(-1)] = torch.arange(T * K, device=y.device)
    pair = pair[:rows]
    w = torch.cat([s["w"].reshape(-1), torch.zeros(1, device=y.device)])
    dy = (w[pair][:, None] * dout[(pair // K).clamp_max(T - 1)]).to(BF16)
    dy = torch.where((pair < T * K)[:, None], dy, s["dy"].view(rows, -1))
    return dy.view(s["dy"].shape), dw


def _act(name, z):
    if name == "relu":
        return torch.where(z > 0, z, 0.0)
    if name == "silu":
        return z / (1 + torch.exp(-z))
    if name == "gelu":
        return 0.5 * z * (1 + torch.erf(z * math.sqrt(0.5)))
    return z


def _act_grad(name, z):
    if name == "relu":
        return torch.where(z > 0, 1.0, 0.0)
    if name == "silu":
        sig = 1 / (1 + torch.exp(-z))
        return sig * (1 + z * (1 - sig))
    return (0.5 * (1 + torch.erf(z * math.sqrt(0.5)))
            + z * torch.exp(-0.5 * z * z) * (1 / math.sqrt(2 * math.pi)))


def _plain_linear(s):
    c = s["case"]
    z = torch.matmul(s["x"].float(), s["w"].float().T)
    if c["bias"]:
        z = z + s["bias"].float()
    out = _act(c["act"], z)
    if c["residual"]:
        out = out + s["residual"].float()
    return (out.to(BF16), z.to(BF16)) if c["keep"] else out.to(BF16)


def _plain_linear_bwd(s):
    dz = s["dout"].float()
    if s["pre"] is not None:
        dz = dz * _act_grad(s["case"]["act"], s["pre"].float())
    dx = torch.matmul(dz, s["w"].float()).to(BF16)
    return dx, torch.matmul(dz.T, s["x"].float()).to(BF16), dz.sum(0)


# ------------------------------------------------------------------------------------------
# what a pass needs, and its exact results
# ------------------------------------------------------------------------------------------

def work(case):
    T, H, op = case["T"], case["H"], case["op"]
    if op == "linear":
        N = case["N"]
        outs = 1 + case["residual"] + case["keep"]
        return {"bytes": 2 * (T * H + N * H + T * N * outs + N * case["bias"]),
                "flops": 2 * T * N * H}
    if op == "linear_bwd":
        N = case["N"]
        return {"bytes": 2 * (T * H * 2 + N * H * 2 + T * N * (1 + (case["act"] != "none"))) + 4 * N,
                "flops": 4 * T * N * H}
    E, K = case["E"], case["K"]
    pairs = min(T * K, E * case["C"])
    if op == "combine_grad":
        pairs = pairs * 0.98
        return {"bytes": T * H * 2 + pairs * H * 4 + T * K * 16, "flops": pairs * H * 3}
    hit = E * (1 - (1 - K / E) ** T)          # experts that get a row, routes spread evenly
    if op == "gemm":
        N = case["N"]
        return {"bytes": 2 * (hit * N * H + pairs * (H + N)), "flops": 2 * pairs * N * H}
    if op == "gemm_bwd":
        N = case["N"]
        return {"bytes": 2 * hit * N * H + (4 if case["f32"] else 2) * E * N * H
                + 2 * pairs * (2 * H + N), "flops": 4 * pairs * N * H}
    I = case["I"]
    if op == "swiglu":
        return {"bytes": 2 * (hit * 2 * I * H + pairs * (H + I + 2 * I * case["keep"])),
                "flops": 4 * pairs * I * H}
    return {"bytes": 2 * (hit * I * H + E * I * H + pairs * (H + 5 * I)),
            "flops": 4 * pairs * I * H}


def _exact_linear(s):
    c = s["case"]
    x, w = s["x"].double(), s["w"].double()
    if c["op"] == "linear":
        z = x @ w.T + (s["bias"].double() if c["bias"] else 0)
        out = {"none": lambda: z, "relu": lambda: z.clamp_min(0), "silu": lambda: z * z.sigmoid(),
               "gelu": lambda: z * torch.special.ndtr(z)}[c["act"]]()
        if c["residual"]:
            out = out + s["residual"].double()
        return (out, z) if c["keep"] else out
    dz = s["dout"].double()
    if s["pre"] is not None:
        with torch.enable_grad():
            z = s["pre"].double().requires_grad_()
            a = {"relu": lambda: z.clamp_min(0), "silu": lambda: z * z.sigmoid(),
                 "gelu": lambda: z * torch.special.ndtr(z)}[c["act"]]()
            if c["act"] == "relu":
                dz = dz * (z.detach() > 0)
            else:
                dz, = torch.autograd.grad(a, z, dz)
    return dz @ w, dz.T @ x, dz.sum(0)


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op in ("linear", "linear_bwd"):
        return _exact_linear(s)
    E, H = case["E"], case["H"]
    if op == "combine_grad":
        dy = s["dy"].double().view(-1, H)
        y = s["y"].view(-1, H)
        dw = torch.zeros(s["w"].shape, dtype=torch.float64, device=dy.device)
        for j in range(case["K"]):
            t = torch.nonzero(s["slot"][:, j] >= 0)[:, 0]
            e = s["idx"][t, j].long()
            r = (s["offset"][e].long() if case["packed"] else e * case["C"]) + s["slot"][t, j]
            d = s["dout"][t].double()
            dy[r] = s["w"][t, j].double()[:, None] * d
            dw[t, j] = (d * y[r].double()).sum(1)
        return dy.view(s["dy"].shape), dw
    count = s["count"].tolist()
    start = s["offset"].tolist() if case["packed"] else [e * case["C"] for e in range(E)]
    flat = {k: v.flatten(0, -2) for k, v in s.items()
            if k in ("x", "y", "dy", "dx", "h", "gu", "dgu") and v is not None}
    out = {k: torch.zeros(v.shape, dtype=torch.float64, device=v.device)
           for k, v in flat.items() if k in ("y", "dx", "h", "gu", "dgu")}
    dw = None
    if op in ("gemm_bwd", "swiglu_bwd"):
        like = s["dw"] if op == "gemm_bwd" else s["dw2"]
        dw = torch.zeros(like.shape, dtype=torch.float64, device=like.device)
    for e in range(E):
        r = slice(start[e], start[e] + count[e])
        if op == "gemm":
            out["y"][r] = flat["x"][r].double() @ s["w"][e].double().T
        elif op == "gemm_bwd":
            d = flat["dy"][r].double()
            out["dx"][r] = d @ s["w"][e].double()
            dw[e] = d.T @ flat["x"][r].double()
        elif op == "swiglu":
            v = flat["x"][r].double() @ s["w13"][e].double().T
            gate, up = v.split(case["I"], 1)
            out["h"][r] = gate * torch.sigmoid(gate) * up
            if case["keep"]:
                out["gu"][r] = v
        else:
            d = flat["dy"][r].double()
            dh = d @ s["w2"][e].double()
            with torch.enable_grad():
                gu = flat["gu"][r].double().requires_grad_()
                gate, up = gu.split(case["I"], 1)
                out["dgu"][r], = torch.autograd.grad(gate * torch.sigmoid(gate) * up, gu, dh)
            dw[e] = d.T @ flat["h"][r].double()
    if op == "gemm":
        return out["y"].view(s["y"].shape)
    if op == "gemm_bwd":
        return out["dx"].view(s["dx"].shape), dw
    if op == "swiglu":
        h = out["h"].view(s["h"].shape)
        return (h, out["gu"].view(s["gu"].shape)) if case["keep"] else h
    return out["dgu"].view(s["dgu"].shape), dw
