"""Outputs and workspaces that a call on another stream allocates: they are memory of that stream,
whose allocator hands a block out in the stream's own order. A block of the current stream may have
a kernel of its last owner still to come, which the call's stream does not wait for."""
import pytest
import torch

from combine_ep_layout_06_amd import binding as B

pytestmark = pytest.mark.gpu

DEV = "cuda"
T, H, E, K, C, R, I = 8, 256, 4, 2, 8, 2, 128


def bf16(*s):
    return torch.zeros(s, dtype=torch.bfloat16, device=DEV)


def i32(*s):
    return torch.zeros(s, dtype=torch.int32, device=DEV)


def u8(*s):
    return torch.zeros(s, dtype=torch.uint8, device=DEV)


def f32(*s):
    return torch.zeros(s, device=DEV)


CALLS = {
    "layout": lambda s: B.ep_layout(i32(T, K), E, C, R, stream=s),
    "layout_dispatch": lambda s: B.ep_layout_dispatch(bf16(T, H), i32(T, K), bf16(E, C, H), E, C, R,
                                                      stream=s),
    "layout_packed": lambda s: B.ep_layout_packed(i32(T, K), E, C, R, 1, stream=s),
    "layout_dispatch_packed": lambda s: B.ep_layout_dispatch_packed(bf16(T, H), i32(T, K),
                                                                    bf16(16, H), E, C, R, 1, stream=s),
    "combine": lambda s: B.ep_combine(bf16(E, C, H), i32(T, K), i32(T, K), f32(T, K), C, stream=s),
    "rank_layout": lambda s: B.ep_rank_layout(i32(T, K), E, R, stream=s),
    "gemm": lambda s: B.ep_expert_gemm_fp8(u8(E, C, H), f32(E, C, 2), i32(E), u8(E, I, H),
                                           f32(E, 1, 2), T * K, stream=s),
    "gemm_packed": lambda s: B.ep_expert_gemm_fp8_packed(u8(16, H), f32(16, 2), i32(E), i32(E + 1),
                                                         u8(E, I, H), f32(E, 1, 2), T * K, stream=s),
    "swiglu": lambda s: B.ep_expert_swiglu_fp8(u8(E, C, H), f32(E, C, 2), i32(E), u8(E, 2 * I, H),
                                               f32(E, 2, 2), T * K, stream=s),
    "swiglu_packed": lambda s: B.ep_expert_swiglu_fp8_packed(
        u8(16, H), f32(16, 2), i32(E), i32(E + 1), u8(E, 2 * I, H), f32(E, 2, 2), T * K, stream=s),
    "layer": lambda s: B.ep_moe_layer(bf16(T, H), i32(T, K), f32(T, K), bf16(E, 2 * I, H),
                                      bf16(E, H, I), stream=s),
    "layer_fp8": lambda s: B.ep_moe_layer_fp8(bf16(T, H), i32(T, K), f32(T, K), u8(E, 2 * I, H),
                                              f32(E, 2, 2), u8(E, H, I), f32(E, 2, 1), stream=s),
}


@pytest.mark.parametrize("call", sorted(CALLS))
def test_missing_outputs_are_memory_of_the_calls_stream(call, monkeypatch):
    """Nothing is launched here."""
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    B.load_library()
    used = []
    empty = torch.empty
    other = torch.cuda.Stream()
    monkeypatch.setattr(B, "_call", lambda *a, **kw: None)
    monkeypatch.setattr(torch, "empty",
                        lambda *a, **kw: (used.append(torch.cuda.current_stream()), empty(*a, **kw))[1])
    CALLS[call](other)
    assert used and all(s == other for s in used), used
    used.clear()
    CALLS[call](None)
    assert used and all(s == torch.cuda.current_stream() for s in used)


def test_an_output_is_not_reused_while_the_current_stream_reads_it():
    """An output of a call on another stream, released while the current stream has work on it to
    come: the next call on that stream does not get its memory."""
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    idx = torch.randint(0, E, (64, K), dtype=torch.int32, device=DEV)
    none = torch.full_like(idx, -1)
    torch.cuda.synchronize()
    other = torch.cuda.Stream()
    want = B.ep_layout(idx, E, 64, R)["slot"].clone()
    torch.cuda.synchronize()
    lay = B.ep_layout(idx, E, 64, R, stream=other)
    torch.cuda.current_stream().wait_stream(other)
    torch.cuda._sleep(20_000_000)                # about 10 ms
    kept = lay["slot"] + 0                       # reads it after that
    del lay
    for _ in range(4):
        B.ep_layout(none, E, 64, R, stream=other)
    torch.cuda.synchronize()
    assert torch.equal(kept, want)
