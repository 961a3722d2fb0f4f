"""The expert operators between dispatch and combine, as measured cases.

Three operators of a mixture-of-experts layer on one GPU:

* ``gemm``    the experts' product on FP8 rows: ``y = (q * scale) @ (w_q * w_scale)^T`` for the
              rows of each expert, scales per row and 128 channels (as the FP8 dispatch writes
              them) and per 128 x 128 block of the weights; y in bf16.
* ``swiglu``  the same product with the gate and up weights, then ``h = silu(g) * u`` and its FP8
              cast (E4M3 codes and one scale per row and 128 channels).
* ``layer``   a whole layer for a few tokens, from bf16 token rows, expert ids and weights to the
              combined bf16 rows: ``out = sum_j w_j * W2[e_j] (silu(Wg[e_j] x) * (Wu[e_j] x))``,
              with bf16 weights or FP8 ones.

``gemm`` and ``swiglu`` take the padded receive buffer [E][C] or the packed one [rows], and leave
rows that hold no pair as they were.

With ``own`` false, ``run`` computes them with elementary torch operations in 32 bits; with ``own``
true it calls the library. ``exact`` computes them in 64 bits.
"""
import math

import torch
import torch.nn.functional as F

own = False

BLOCK = 128
E4M3 = torch.float8_e4m3fn
LAYER_PAIRS = 1024        # most (token, expert) pairs of a drawn layer case


def listed():
    return [
        # the down projection of the FP8 prefill workload (4096 tokens, 96 experts, top-8),
        # capacity 512: the padded receive buffer, every expert's rows end inside a tile
        dict(name="gemm_prefill", op="gemm", packed=False, T=4096, E=96, K=8, H=768, N=2048, C=512,
             A=1, route="uniform"),
        # the same projection in a decode step of 128 tokens: 8 rows an expert, all weights read
        dict(name="gemm_decode", op="gemm", packed=False, T=128, E=128, K=8, H=768, N=2048, C=128,
             A=1, route="uniform"),
        # a small, skewed batch in the packed layout with no alignment and an odd output width
        dict(name="gemm_ragged", op="gemm", packed=True, T=777, E=32, K=4, H=640, N=1000, C=777,
             A=1, route="zipf"),
        # a long prefill on few, large experts (one GPU's 32): bound by the matrix units
        dict(name="gemm_large", op="gemm", packed=True, T=8192, E=32, K=8, H=4096, N=4096, C=2560,
             A=128, route="uniform"),
        # gate and up of the FP8 prefill workload
        dict(name="swiglu_prefill", op="swiglu", packed=False, T=4096, E=96, K=8, H=2048, I=768,
             C=512, A=1, route="uniform"),
        # gate and up of a decode step in the packed layout, routing skewed
        dict(name="swiglu_decode", op="swiglu", packed=True, T=128, E=128, K=8, H=2048, I=768,
             C=128, A=16, route="zipf"),
        # gate and up of a long prefill on one GPU's 32 large experts
        dict(name="swiglu_large", op="swiglu", packed=True, T=8192, E=32, K=8, H=4096, I=2048,
             C=2560, A=128, route="uniform"),
        # one token generated alone: the smallest call, where latency counts
        dict(name="layer_bf16_1", op="layer", fp8=False, T=1, E=128, K=8, H=2048, I=768,
             route="uniform"),
        # a decode step of 32 sequences with bf16 weights
        dict(name="layer_bf16_32", op="layer", fp8=False, T=32, E=128, K=8, H=2048, I=768,
             route="uniform"),
        # one token with FP8 weights: half the bytes
        dict(name="layer_fp8_1", op="layer", fp8=True, T=1, E=128, K=8, H=2048, I=768,
             route="uniform"),
        # a few sequences (a speculative step), skewed routing
        dict(name="layer_fp8_12", op="layer", fp8=True, T=12, E=96, K=8, H=2048, I=768,
             route="zipf"),
        # the decode workload's 128 tokens: every expert's weights are read
        dict(name="layer_fp8_128", op="layer", fp8=True, T=128, E=128, K=8, H=2048, I=768,
             route="uniform"),
    ]


def _log(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def _blocks(rng, lo, hi, step):
    return step * _log(rng, lo // step, hi // step)


def draw(rng):
    op = rng.choice(("gemm", "swiglu", "layer"))
    E = _log(rng, 1, 160)
    K = rng.randint(1, min(8, E))
    route = rng.choice(("uniform", "zipf"))
    if op == "layer":
        fp8 = rng.random() < 0.5
        step = 128 if fp8 else 64
        H, I = _blocks(rng, 256, 4096, step), _blocks(rng, 128, 2048, step)
        T = _log(rng, 1, LAYER_PAIRS // K)
        while E * H * I > 128 * 2048 * 768:
            E = max(K, E // 2)
            if E == K:
                I = max(step, I // 2 // step * step)
        return dict(op=op, fp8=fp8, T=T, E=E, K=K, H=H, I=I, route=route)
    H = _blocks(rng, 128, 4096, 128)
    T = _log(rng, 1, 8192)
    if op == "gemm":
        N = 8 * _log(rng, 8, 512)
    else:
        I = _blocks(rng, 128, 2048, 128)
        N = 2 * I
    while E * H * N > 128 * 2048 * 2048:
        E = max(K, E // 2)
        if E == K:
            break
    C = min(T, int(1.25 * T * K / E) + 16)
    while E * C * H * N > 32 * 2560 * 4096 * 4096:
        T = max(1, T // 2)
        C = min(T, int(1.25 * T * K / E) + 16)
    packed = rng.random() < 0.5
    A = rng.choice((1, 16, 24, 128)) if packed else 1
    c = dict(op=op, packed=packed, T=T, E=E, K=K, H=H, C=C, A=A, route=route)
    return dict(c, N=N) if op == "gemm" else dict(c, I=I)


# ------------------------------------------------------------------------------------------
# inputs
# ------------------------------------------------------------------------------------------

def _route(case, g, dev):
    """K distinct experts for each token, uniformly or by a Zipf(1.2) law over a random order."""
    T, E, K = case["T"], case["E"], case["K"]
    keys = -torch.log(-torch.log(torch.rand(T, E, generator=g, device=dev, dtype=torch.float64)))
    if case["route"] == "zipf":
        rank = torch.randperm(E, generator=g, device=dev)
        keys = keys - 1.2 * torch.log(rank + 1.0)
    return torch.argsort(keys, dim=1, descending=True)[:, :K].to(torch.int32).contiguous()


def _tokens(n, H, g, dev):
    """bf16 rows, N(0, 1) with one channel value in a hundred 50 times larger."""
    x = torch.randn(n, H, generator=g, device=dev)
    big = torch.rand(n, H, generator=g, device=dev) < 0.01
    return torch.where(big, 50 * x, x).to(torch.bfloat16)


def _quantise_rows(x):
    """E4M3 codes and fp32 scales (amax / 448) per row and 128 channels."""
    b = x.float().unflatten(-1, (-1, BLOCK))
    s = b.abs().amax(-1) / 448
    q = (b / s.clamp_min(1e-30)[..., None]).clamp(-448, 448).to(E4M3)
    return q.flatten(-2), s


def _quantise_weights(E, N, H, g, dev):
    """E4M3 codes [E, N, H] and scales [E, ceil(N / 128), H / 128] of random weights whose
    spread differs from block to block."""
    nb, hb = -(-N // BLOCK), H // BLOCK
    q = torch.empty(E, N, H, dtype=E4M3, device=dev)
    s = torch.empty(E, nb, hb, device=dev)
    some = max(1, (1 << 28) // (nb * BLOCK * H))
    for e in range(0, E, some):
        n = min(some, E - e)
        spread = torch.exp(0.5 * torch.randn(n, nb, hb, generator=g, device=dev)) / math.sqrt(H)
        w = torch.randn(n, nb, BLOCK, hb, BLOCK, generator=g, device=dev)
        w *= spread[:, :, None, :, None]
        sc = w.abs().amax((2, 4)) / 448
        w /= sc[:, :, None, :, None]
        q[e:e + n] = w.clamp_(-448, 448).reshape(n, nb * BLOCK, H)[:, :N].to(E4M3)
        s[e:e + n] = sc
    return q, s


def _layout(case, idx):
    """Slots in token order under the capacity, counts, and the packed offsets."""
    E, C, A = case["E"], case["C"], case["A"]
    flat = idx.reshape(-1).long()
    seen = F.one_hot(flat, E).cumsum(0)
    slot = seen.gather(1, flat[:, None])[:, 0] - 1
    count = torch.bincount(flat, minlength=E).clamp_max(C)
    padded = (count + A - 1) // A * A
    offset = torch.cat([torch.zeros(1, dtype=torch.long, device=idx.device), padded.cumsum(0)])
    return flat, slot, slot < C, count.to(torch.int32), offset.to(torch.int32)


def prepare(case, seed):
    dev = torch.device("cuda", torch.cuda.current_device())
    g = torch.Generator(device=dev)
    g.manual_seed(seed)
    T, E, K, H = case["T"], case["E"], case["K"], case["H"]
    idx = _route(case, g, dev)
    x = _tokens(T, H, g, dev)
    s = dict(case=case, pairs=T * K)
    if case["op"] == "layer":
        I = case["I"]
        s.update(x=x, topk_idx=idx)
        s["topk_w"] = torch.softmax(torch.randn(T, K, generator=g, device=dev), 1)
        for name, n, k in (("w13", 2 * I, H), ("w2", H, I)):
            if case["fp8"]:
                s[name], s[name + "_scale"] = _quantise_weights(E, n, k, g, dev)
            else:
                w = torch.empty(E, n, k, dtype=torch.bfloat16, device=dev)
                s[name] = w.normal_(0, 1 / math.sqrt(k), generator=g)
        s["out"] = torch.zeros(T, H, dtype=torch.bfloat16, device=dev)
        # a workspace for the largest step of a serving loop: enough for any of these
        s["workspace"] = torch.empty(8 * T * K * (I + H) + (1 << 20), dtype=torch.uint8, device=dev)
        return s
    N = case["N"] if case["op"] == "gemm" else 2 * case["I"]
    flat, slot, kept, count, offset = _layout(case, idx)
    q, sc = _quantise_rows(x)
    if case["packed"]:
        rows = min(T * K, E * case["C"]) + E * (case["A"] - 1)
        at = offset[flat].long() + slot
        s["packed_offset"] = offset
        lead = (rows,)
    else:
        at = flat * case["C"] + slot
        lead = (E, case["C"])
        rows = E * case["C"]
    at, token = at[kept], torch.arange(T * K, device=dev)[kept] // K
    recv_q = torch.zeros(rows, H, dtype=torch.uint8, device=dev)
    recv_scale = torch.zeros(rows, H // BLOCK, device=dev)
    recv_q[at] = q.view(torch.uint8)[token]
    recv_scale[at] = sc[token]
    s["recv_q"] = recv_q.view(E4M3).reshape(*lead, H)
    s["recv_scale"] = recv_scale.reshape(*lead, H // BLOCK)
    s["expert_count"] = count
    s["w_q"], s["w_scale"] = _quantise_weights(E, N, H, g, dev)
    if case["op"] == "gemm":
        s["y"] = torch.zeros(*lead, N, dtype=torch.bfloat16, device=dev)
    else:
        s["h_q"] = torch.zeros(*lead, case["I"], dtype=torch.uint8, device=dev).view(E4M3)
        s["h_scale"] = torch.zeros(*lead, case["I"] // BLOCK, device=dev)
    return s


# ------------------------------------------------------------------------------------------
# the operators
# ------------------------------------------------------------------------------------------

def run(state):
    op = state["case"]["op"]
    if op == "gemm":
        return _own_gemm(state) if own else _plain_gemm(state)
    if op == "swiglu":
        return _own_swiglu(state) if own else _plain_swiglu(state)
    return _own_layer(state) if own else _plain_layer(state)


def _own_gemm(s):
    from combine_ep_layout_06_amd import binding as B
    if s["case"]["packed"]:
        return B.ep_expert_gemm_fp8_packed(s["recv_q"], s["recv_scale"], s["expert_count"],
                                           s["packed_offset"], s["w_q"], s["w_scale"], s["pairs"],
                                           y=s["y"])
    return B.ep_expert_gemm_fp8(s["recv_q"], s["recv_scale"], s["expert_count"], s["w_q"],
                                s["w_scale"], s["pairs"], y=s["y"])


def _own_swiglu(s):
    from combine_ep_layout_06_amd import binding as B
    if s["case"]["packed"]:
        return B.ep_expert_swiglu_fp8_packed(s["recv_q"], s["recv_scale"], s["expert_count"],
                                             s["packed_offset"], s["w_q"], s["w_scale"],
                                             s["pairs"], h_q=s["h_q"], h_scale=s["h_scale"])
    return B.ep_expert_swiglu_fp8(s["recv_q"], s["recv_scale"], s["expert_count"], s["w_q"],
                                  s["w_scale"], s["pairs"], h_q=s["h_q"], h_scale=s["h_scale"])


def _own_layer(s):
    from combine_ep_layout_06_amd import binding as B
    if s["case"]["fp8"]:
        return B.ep_moe_layer_fp8(s["x"], s["topk_idx"], s["topk_w"], s["w13"], s["w13_scale"],
                                  s["w2"], s["w2_scale"], out=s["out"], workspace=s["workspace"])
    return B.ep_moe_layer(s["x"], s["topk_idx"], s["topk_w"], s["w13"], s["w2"], out=s["out"],
                          workspace=s["workspace"])


def _rows_f32(q, scale):
    return (q.float().unflatten(-1, (-1, BLOCK)) * scale[..., None]).flatten(-2)


def _weights_f32(q, scale):
    per_row = scale.repeat_interleave(BLOCK, dim=1)[:, :q.shape[1]]
    return (q.float().unflatten(-1, (-1, BLOCK)) * per_row[..., None]).flatten(-2)


def _product(s):
    """The experts' products of all rows in 32 bits, [E, C, N] whatever the layout."""
    c = s["case"]
    x = _rows_f32(s["recv_q"], s["recv_scale"])
    if c["packed"]:
        at = s["packed_offset"][:-1, None].long() + torch.arange(c["C"], device=x.device)
        x = x[at.clamp_max(x.shape[0] - 1)]
    return torch.matmul(x, _weights_f32(s["w_q"], s["w_scale"]).transpose(1, 2))


def _place(s, v, before):
    """v [E, C, n] where a pair's row is, `before` elsewhere."""
    c = s["case"]
    if not c["packed"]:
        held = torch.arange(c["C"], device=v.device) < s["expert_count"][:, None]
        return torch.where(held[..., None], v, before)
    row = torch.arange(before.shape[0], device=v.device, dtype=torch.int32)
    e = torch.searchsorted(s["packed_offset"][1:], row, right=True).clamp_max(c["E"] - 1)
    slot = row - s["packed_offset"][e]
    held = slot < s["expert_count"][e]
    return torch.where(held[:, None], v[e, slot.clamp(0, c["C"] - 1).long()], before)


def _plain_gemm(s):
    return _place(s, _product(s).to(torch.bfloat16), s["y"])


def _plain_swiglu(s):
    gate, up = _product(s).chunk(2, -1)
    h = (gate / (1 + torch.exp(-gate)) * up).unflatten(-1, (-1, BLOCK))
    scale = h.abs().amax(-1) / 448
    q = (h / scale.clamp_min(1e-38)[..., None]).clamp(-448, 448).flatten(-2).to(E4M3)
    q = _place(s, q.view(torch.uint8), s["h_q"].view(torch.uint8)).view(E4M3)
    return q, _place(s, scale, s["h_scale"])


def _layer_weights(s, which, e=None):
    w = s[which] if e is None else s[which].view(torch.uint8)[e].view(E4M3) if s["case"]["fp8"] \
        else s[which][e]
    if not s["case"]["fp8"]:
        return w.float()
    return _weights_f32(w, s[which + "_scale"] if e is None else s[which + "_scale"][e])


def _plain_layer(s):
    c = s["case"]
    T, E, K = c["T"], c["E"], c["K"]
    x, idx = s["x"].float(), s["topk_idx"].long()
    if T * K <= E:           # the chosen experts' weights, pair by pair
        e = idx.reshape(-1)
        rows = x.repeat_interleave(K, 0)[:, None]
        gate, up = torch.matmul(rows, _layer_weights(s, "w13", e).transpose(1, 2)).chunk(2, -1)
        h = gate / (1 + torch.exp(-gate)) * up
        y = torch.matmul(h, _layer_weights(s, "w2", e).transpose(1, 2)).view(T, K, -1)
    else:                    # every expert on every token
        gate, up = torch.matmul(x, _layer_weights(s, "w13").transpose(1, 2)).chunk(2, -1)
        h = gate / (1 + torch.exp(-gate)) * up
        y = torch.matmul(h, _layer_weights(s, "w2").transpose(1, 2))
        y = y[idx, torch.arange(T, device=x.device)[:, None]]
    return (s["topk_w"][..., None] * y).sum(1).to(torch.bfloat16)


# ------------------------------------------------------------------------------------------
# what a pass needs, and its exact results
# ------------------------------------------------------------------------------------------

def work(case):
    T, E, K, H = case["T"], case["E"], case["K"], case["H"]
    pairs = T * K
    hit = E * (1 - (1 - K / E) ** T)          # experts that get a row, routes spread evenly
    if case["op"] == "layer":
        I = case["I"]
        size = 1 + 4 / BLOCK ** 2 if case["fp8"] else 2
        return {"bytes": hit * 3 * I * H * size + T * H * 4 + pairs * 8,
                "flops": pairs * 6 * I * H}
    N = case["N"] if case["op"] == "gemm" else 2 * case["I"]
    out = 2 * N if case["op"] == "gemm" else case["I"] * (1 + 4 / BLOCK)
    return {"bytes": hit * N * H * (1 + 4 / BLOCK ** 2) + pairs * (H * (1 + 4 / BLOCK) + out),
            "flops": pairs * 2 * N * H}


def _f64(q, scale, rows):
    """One matrix of codes in 64 bits, its scale for each `rows` x 128 block."""
    q = q.to(torch.float64)
    full = torch.kron(scale.double(), torch.ones(rows, BLOCK, dtype=torch.float64, device=q.device))
    return q * full[:q.shape[0]]


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "layer":
        x, out = s["x"].double(), torch.zeros(s["x"].shape, dtype=torch.float64, device=s["x"].device)
        for e in torch.unique(s["topk_idx"]).tolist():
            t, j = torch.nonzero(s["topk_idx"] == e, as_tuple=True)
            if case["fp8"]:
                w13, w2 = (_f64(s[n][e], s[n + "_scale"][e], BLOCK) for n in ("w13", "w2"))
            else:
                w13, w2 = s["w13"][e].double(), s["w2"][e].double()
            gate, up = (x[t] @ w13.T).split(case["I"], 1)
            y = (gate * torch.sigmoid(gate) * up) @ w2.T
            out.index_add_(0, t, s["topk_w"][t, j].double()[:, None] * y)
        return out
    count = s["expert_count"].tolist()
    gemm = case["op"] == "gemm"
    lead = s["recv_q"].shape[:-1]
    q, scale = s["recv_q"].flatten(0, -2), s["recv_scale"].flatten(0, -2)
    n = case["N"] if gemm else case["I"]
    out = torch.zeros(q.shape[0], n, dtype=torch.float64, device=q.device)
    hs = None if gemm else torch.zeros(q.shape[0], n // BLOCK, dtype=torch.float64, device=q.device)
    start = s["packed_offset"].tolist() if case["packed"] else [e * case["C"] for e in range(case["E"])]
    for e in range(case["E"]):
        r = slice(start[e], start[e] + count[e])
        y = _f64(q[r], scale[r], 1) @ _f64(s["w_q"][e], s["w_scale"][e], BLOCK).T
        if gemm:
            out[r] = y
            continue
        h = y[:, :n] * torch.sigmoid(y[:, :n]) * y[:, n:]
        sc = h.view(-1, n // BLOCK, BLOCK).abs().amax(-1) / 448
        hs[r] = sc
        out[r] = h / sc.clamp_min(1e-300).repeat_interleave(BLOCK, 1)
    if gemm:
        return out.view(*lead, n)
    return out.view(*lead, n), hs.view(*lead, n // BLOCK)
