"""Calls on a stream that is not the current one: what a call allocates (results, workspaces) belongs to the stream that
uses it, so that new allocations of the current stream cannot take the memory while the call is still to run."""
import numpy as np
import pytest
import torch

import block_quantized_bit_amd as q4

pytestmark = pytest.mark.gpu


def rand(seed, *shape, dtype=torch.float32):
    return torch.from_numpy(np.random.default_rng(seed).standard_normal(shape).astype(np.float32)).cuda().to(dtype)


def i32(values):
    return torch.tensor(values, dtype=torch.int32, device="cuda")


def stream_of_memory(t):
    """Handle of the stream whose memory the allocator gave to t."""
    for segment in torch.cuda.memory_snapshot():
        if segment["address"] <= t.data_ptr() < segment["address"] + segment["total_size"]:
            return segment["stream"]
    raise AssertionError("not the allocator's memory")


def e4m3_calls():
    x, dy = rand(0, 300, 512, dtype=torch.bfloat16), rand(1, 300, 200, dtype=torch.bfloat16)
    wq, ws = q4.f8_quantize_weights(rand(2, 200, 512))
    wqt, wst = q4.f8_transpose_weights(wq, ws, 512)
    xq, xs = q4.f8_quantize_act(x)
    w = rand(2, 200, 512)
    return {
        "f8_linear": lambda **kw: [q4.f8_linear(x, wq, ws, **kw)],
        "f8_linear_backward": lambda **kw: q4.f8_linear_backward(dy, x, wqt, wst, **kw),
        "f8_gemm": lambda **kw: [q4.f8_gemm(xq, xs, wq, ws, **kw)],
        "f8_quantize_act": lambda **kw: q4.f8_quantize_act(x, **kw),
        "f8_quantize_act_t": lambda **kw: q4.f8_quantize_act_t(x, **kw),
        "f8_quantize_weights": lambda **kw: q4.f8_quantize_weights(w, **kw),
        "f8_transpose_weights": lambda **kw: q4.f8_transpose_weights(wq, ws, 512, **kw),
    }


def cache_calls():
    n, heads, d = 3000, 2, 64
    cache = q4.kv8_cache(50, heads, 64, d)
    table, length, one, whole = i32([list(range(50))]), i32([n]), i32([0, 1]), i32([0, n])
    q4.kv8_append(rand(3, n, heads, d), rand(4, n, heads, d), *cache, table, length, whole, n)
    q = rand(5, 1, 8, d)
    return {
        "kv8_attention": lambda **kw: [q4.kv8_attention(q, *cache, table, length, one, 1, n, **kw)],  # in splits
        "kv8_read": lambda **kw: q4.kv8_read(*cache, table, length, whole, n, total=n, **kw),
    }


def mlp_calls():
    x, logits = rand(6, 5, 256), rand(7, 5, 4)
    up = [q4.quantize_weights(rand(8 + e, 256, 256), "q4_0", 32) for e in range(4)]
    down = [q4.quantize_weights(rand(18 + e, 256, 128), "q4_0", 32) for e in range(4)]
    w13, s13, w2, s2 = (torch.stack([w[i] for w in ws]) for ws in (up, down) for i in range(2))
    return {"moe_q4": lambda **kw: [q4.moe_q4(x, logits, w13, s13, None, w2, s2, None, 2, **kw)]}


def check(call):
    """The call on a side stream that is busy, while the current stream allocates and overwrites: same bits as on the
    current stream, results in the side stream's memory."""
    want = [t.clone() for t in call()]
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        torch.cuda._sleep(10_000_000)  # some milliseconds, in which the call waits
    got = call(stream=side)
    handle = side.cuda_stream
    assert torch.cuda.current_stream().cuda_stream != handle  # as it was before the call
    # blocks of every size class, several of each, all overwritten before the call can run
    junk = [torch.empty(1 << size, dtype=torch.uint8, device="cuda").fill_(255) for size in range(9, 25) for _ in range(6)]
    torch.cuda.synchronize()
    del junk
    for g, w in zip(got, want):
        assert stream_of_memory(g) == handle
        assert torch.equal(g.view(torch.uint8), w.view(torch.uint8))


@pytest.mark.parametrize("name", ["f8_linear", "f8_linear_backward", "f8_gemm", "f8_quantize_act", "f8_quantize_act_t",
                                  "f8_quantize_weights", "f8_transpose_weights"])
def test_e4m3_product(name):
    check(e4m3_calls()[name])


@pytest.mark.parametrize("name", ["kv8_attention", "kv8_read"])
def test_cache(name):
    check(cache_calls()[name])


def test_routed_mlp():
    check(mlp_calls()["moe_q4"])


def test_streams_by_handle_and_under_a_context():
    """An object that only has a handle, the default stream, and the current stream's own handle."""
    class Handle:
        def __init__(self, stream):
            self.cuda_stream = stream.cuda_stream

    side = torch.cuda.Stream()
    x = rand(0, 100, 256)
    wq, ws = q4.f8_quantize_weights(rand(1, 64, 256))
    want = q4.f8_linear(x, wq, ws)
    torch.cuda.synchronize()
    for given in (Handle(side), side, torch.cuda.default_stream(), torch.cuda.current_stream()):
        y = q4.f8_linear(x, wq, ws, stream=given)
        xq, _ = q4.f8_quantize_act(x, stream=given)
        torch.cuda.synchronize()
        assert torch.equal(y, want)
        assert stream_of_memory(y) == stream_of_memory(xq) == given.cuda_stream
    with torch.cuda.stream(side):
        y = q4.f8_linear(x, wq, ws, stream=torch.cuda.default_stream())
        assert torch.cuda.current_stream() == side
        torch.cuda.synchronize()
        assert stream_of_memory(y) == torch.cuda.default_stream().cuda_stream and torch.equal(y, want)
    with pytest.raises(AttributeError):
        q4.f8_linear(x, wq, ws, stream=7)


def matmul_calls():
    x = rand(30, 40, 512)
    wq, wd, _ = q4.quantize_weights(rand(31, 256, 512), "q4_0", 32)
    act, one = q4.quantize_act(x, 32), q4.quantize_act(x[:1], 32)
    aq, ascale, abias = q4.quantize_weights(rand(32, 256, 512), "affine", 128)
    packed = q4.pack_weights("affine", 128, aq, ascale, abias)
    blocks, w, dy = q4.q4k_quantize_weights(rand(33, 256, 512)), rand(34, 256, 512), rand(35, 16, 256)
    return {
        "quantize_act": lambda **kw: q4.quantize_act(x, 32, **kw),
        "gemv": lambda **kw: [q4.gemv("q4_0", 32, wq, wd, None, *one, **kw)],
        "gemv_fused": lambda **kw: [q4.gemv_fused("q4_0", 32, x[:1], wq, wd, None, **kw)],
        "gemm": lambda **kw: [q4.gemm("q4_0", 32, wq, wd, None, *act, **kw)],
        "pack_weights": lambda **kw: [q4.pack_weights("affine", 128, aq, ascale, abias, **kw)],
        "gemm_packed": lambda **kw: [q4.gemm_packed("affine", 128, x, packed, 256, **kw)[0]],
        "q4k_gemv": lambda **kw: [q4.q4k_gemv(blocks, x[:1], 256, **kw)],
        "q4k_gemm": lambda **kw: [q4.q4k_gemm(blocks, x, 256, **kw)],
        "q4k_gemm_work": lambda **kw: [q4.q4k_gemm_work(blocks, x, 256, **kw)],
        "q4k_gemm_backward": lambda **kw: [q4.q4k_gemm_backward(blocks, dy, 512, **kw)],
        "gemm_backward": lambda **kw: [q4.gemm_backward("q4_0", 32, wq, wd, None, dy, **kw)],
        "quantize_weights": lambda **kw: q4.quantize_weights(w, "q4_0", 32, **kw)[:2],
        "q4k_quantize_weights": lambda **kw: [q4.q4k_quantize_weights(w, **kw)],
    }


@pytest.mark.parametrize("name", ["quantize_act", "gemv", "gemv_fused", "gemm", "pack_weights", "gemm_packed", "q4k_gemv",
                                  "q4k_gemm", "q4k_gemm_work", "q4k_gemm_backward", "gemm_backward",
                                  "quantize_weights", "q4k_quantize_weights"])
def test_4_bit_products(name):
    check(matmul_calls()[name])
