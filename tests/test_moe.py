"""The routed MLP on 4-bit experts on the GPU against 64-bit values on the CPU (tests/_wide.py, moe: the bound follows
the float32 steps and allows a hidden code to differ only where its quotient is within its own error of a half)."""
import numpy as np
import pytest
import torch

import block_quantized_bit_amd as q4
from tests import _wide as W

pytestmark = pytest.mark.gpu

FORMATS = [("q4_0", 32), ("affine", 64), ("affine", 128)]


def experts(r, E, N, K, fmt, bs):
    """(codes, scales, biases) on the GPU and their values in float64."""
    c = np.clip(np.round(r.standard_normal((E, N, K)) * 2.6 + 7.5), 0, 15).astype(np.uint8).reshape(E, N, K // 32, 2, 16)
    codes = (c[:, :, :, 0] | (c[:, :, :, 1] << 4)).reshape(E, N, K // 2)
    s = torch.from_numpy((r.uniform(0.6, 1.4, (E, N, K // bs)) * 0.03).astype(np.float32))
    s = s.to(torch.float16 if fmt == "q4_0" else torch.bfloat16)
    b = None if fmt == "q4_0" else (-7.5 * s.float()).to(torch.bfloat16)
    v = W.q4_values(codes, W.as_f64(s), None if b is None else W.as_f64(b), bs)
    return (torch.from_numpy(codes).cuda(), s.cuda(), None if b is None else b.cuda()), v


def layer(r, E, H, inter, fmt, bs):
    (w13, s13, b13), v13 = experts(r, E, 2 * inter, H, fmt, bs)
    (w2, s2, b2), v2 = experts(r, E, H, inter, fmt, bs)
    return (w13, s13, b13, w2, s2, b2), v13, v2


def check(x, logits, weights, v13, v2, k, fmt, bs, renorm=True):
    out = torch.full_like(x, float("nan"))
    got = q4.moe_q4(x, logits, *weights, k, fmt=fmt, bs=bs, renormalize=renorm, out=out)
    y, e = W.moe(W.as_f64(x), W.as_f64(logits), v13, v2, k, bs, renorm)
    if x.dtype == torch.bfloat16:
        e = e + 2.0 ** -8 * (np.abs(y) + e)
    err = np.abs(W.as_f64(got) - y)
    assert (err <= e + 1e-30).all(), (err / (e + 1e-30)).max()
    return got


def inputs(r, T, H, E, dtype):
    x = torch.from_numpy(r.standard_normal((T, H)).astype(np.float32)).cuda().to(dtype)
    return x, torch.from_numpy(r.standard_normal((T, E)).astype(np.float32)).cuda()


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("fmt,bs", FORMATS)
@pytest.mark.parametrize("T,E,k,H,inter", [
    (1, 1, 1, 128, 128), (1, 8, 2, 256, 384), (3, 4, 4, 384, 256), (7, 100, 8, 128, 128), (2, 200, 3, 256, 640),
    (16, 4, 2, 128, 1152), (33, 3, 2, 256, 128), (64, 2, 1, 128, 256), (5, 512, 16, 128, 128),
])
def test_layer(T, E, k, H, inter, fmt, bs, dtype):
    print(f"case moe T={T} E={E} k={k} H={H} I={inter} {fmt} {bs} {dtype}", flush=True)
    r = np.random.default_rng(T + E + H + inter)
    weights, v13, v2 = layer(r, E, H, inter, fmt, bs)
    x, logits = inputs(r, T, H, E, dtype)
    check(x, logits, weights, v13, v2, k, fmt, bs)


def test_wide_rows():
    """H and I of several kilobytes: more than one piece a lane, and token batches cut to the LDS."""
    r = np.random.default_rng(1)
    for H, inter, T in [(4608, 64, 9), (64, 4160, 3), (16384, 64, 8)]:
        print(f"case moe wide {H} {inter}", flush=True)
        weights, v13, v2 = layer(r, 2, H, inter, "q4_0", 32)
        x, logits = inputs(r, T, H, 2, torch.float32)
        check(x, logits, weights, v13, v2, 2, "q4_0", 32)


def test_the_weights_are_those_of_the_library():
    """Experts quantized by quantize_weights, and the layer against its single products."""
    r = np.random.default_rng(2)
    E, H, inter = 2, 256, 128
    w13 = torch.from_numpy((0.05 * r.standard_normal((E, 2 * inter, H))).astype(np.float32)).cuda()
    w2 = torch.from_numpy((0.05 * r.standard_normal((E, H, inter))).astype(np.float32)).cuda()
    a = [q4.quantize_weights(w, "q4_0", 32) for w in w13]
    b = [q4.quantize_weights(w, "q4_0", 32) for w in w2]
    stack = [torch.stack([t[i] for t in a]) for i in range(2)] + [None] + \
            [torch.stack([t[i] for t in b]) for i in range(2)] + [None]
    x, _ = inputs(r, 1, H, E, torch.float32)
    logits = torch.tensor([[1.0, 2.0]], device="cuda")
    got = q4.moe_q4(x, logits, *stack, 1)
    gu = q4.gemv("q4_0", 32, *a[1], *q4.quantize_act(x, 32))
    h = torch.nn.functional.silu(gu[:, :inter]) * gu[:, inter:]
    want = q4.gemv("q4_0", 32, *b[1], *q4.quantize_act(h.contiguous(), 32))
    assert torch.allclose(got, want, rtol=0, atol=2e-3 * float(want.abs().max()))


@pytest.mark.parametrize("renorm", [True, False])
def test_routing(renorm):
    """Ties go to the lower index; -inf and NaN take an expert out; a token with none left gives zeros."""
    r = np.random.default_rng(4)
    E, H, inter = 70, 128, 64
    weights, v13, v2 = layer(r, E, H, inter, "q4_0", 32)
    x, logits = inputs(r, 6, H, E, torch.float32)
    inf, nan = float("inf"), float("nan")
    logits[0] = 0.25
    logits[1] = -inf
    logits[1, 66] = 3.0
    logits[2] = nan
    logits[3, 5:] = logits[3, 4]
    logits[4] = -inf
    logits[4, [3, 64]] = torch.tensor([-80.0, 90.0], device="cuda")
    y = check(x, logits, weights, v13, v2, 3, "q4_0", 32, renorm)
    assert (y[2] == 0).all()


def test_zero_and_large_tokens_repeatability_and_streams():
    r = np.random.default_rng(5)
    weights, v13, v2 = layer(r, 4, 128, 128, "affine", 64)
    x, logits = inputs(r, 5, 128, 4, torch.float32)
    x[0] = 0.0
    x[1] *= 1e-20
    x[2] *= 1e4
    y = check(x, logits, weights, v13, v2, 2, "affine", 64)
    assert (y[0] == 0).all()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        again = q4.moe_q4(x, logits, *weights, 2, fmt="affine", bs=64)
    side.synchronize()
    assert torch.equal(y, again)


def test_refusals():
    r = np.random.default_rng(6)
    weights, _, _ = layer(r, 4, 128, 128, "q4_0", 32)
    x, logits = inputs(r, 2, 128, 4, torch.float32)
    w13, s13, _, w2, s2, _ = weights
    for args, kw in [((x.half(), logits, *weights, 2), {}), ((x, logits.double(), *weights, 2), {}),
                     ((x, logits[:1], *weights, 2), {}), ((x, logits, *weights, 2), dict(bs=48)),
                     ((x, logits, w13, s13.bfloat16(), None, w2, s2, None, 2), {}),
                     ((x, logits, *weights, 2), dict(fmt="q5")), ((x.t(), logits, *weights, 2), {}),
                     ((x, logits, w13, s13, None, w2[:, :, :32], s2, None, 2), {})]:
        with pytest.raises(ValueError):
            q4.moe_q4(*args, **kw)
    for args in [(x, logits, *weights, 5), (x, logits, *weights, 0)]:
        with pytest.raises(q4.Q4Error):
            q4.moe_q4(*args)
    many = torch.zeros(65, 128, device="cuda")
    with pytest.raises(q4.Q4Error):
        q4.moe_q4(many, torch.zeros(65, 4, device="cuda"), *weights, 2)


@pytest.mark.parametrize("bs", [64, 128])
@pytest.mark.parametrize("T,k,blocks", [(64, 16, 1), (64, 16, 3), (64, 16, 4), (64, 16, 6), (64, 16, 7), (56, 16, 6),
                                        (53, 16, 7)])
def test_many_pairs_fill_the_lds(T, k, blocks, bs):
    """Up to 1024 pairs of token and expert, whose sums take 128 KiB: the hidden values' scales (8 bytes a pair and block)
    are staged beside them only where both fit 160 KiB."""
    print(f"case moe pairs T={T} k={k} blocks={blocks} {bs}", flush=True)
    r = np.random.default_rng(T + blocks + bs)
    weights, v13, v2 = layer(r, 20, 128, blocks * bs, "affine", bs)
    x, logits = inputs(r, T, 128, 20, torch.float32)
    check(x, logits, weights, v13, v2, k, "affine", bs)


@pytest.mark.parametrize("aligned", [True, False])
@pytest.mark.parametrize("bs", [64, 128])
@pytest.mark.parametrize("H,inter", [(512, 512), (1024, 1536), (512, 640), (640, 512)])
def test_scales_of_four_steps_in_one_load(H, inter, bs, aligned):
    """Rows of scales that start on 8 or 16 bytes come four steps at a time (H or I a multiple of 512, for each of the
    two products by itself), others one by one: the same layer with scales at an odd offset."""
    print(f"case moe wide scales {H} {inter} {bs} {aligned}", flush=True)
    r = np.random.default_rng(H + inter + bs)
    (w13, s13, b13, w2, s2, b2), v13, v2 = layer(r, 3, H, inter, "affine", bs)
    if not aligned:
        def moved(t):
            return torch.cat([t.new_zeros(1), t.flatten()])[1:].view(t.shape)
        s13, b13, s2, b2 = (moved(t) for t in (s13, b13, s2, b2))
        assert s13.data_ptr() % 16 == 2 and s13.is_contiguous()
    x, logits = inputs(r, 20, H, 3, torch.float32)
    check(x, logits, (w13, s13, b13, w2, s2, b2), v13, v2, 2, "affine", bs)


def test_scales_that_are_not_staged():
    """128 pairs of 128 blocks: 128 KiB of scales and sums of the hidden values, read from memory."""
    r = np.random.default_rng(7)
    weights, v13, v2 = layer(r, 4, 128, 8192, "affine", 64)
    x, logits = inputs(r, 64, 128, 4, torch.float32)
    check(x, logits, weights, v13, v2, 2, "affine", 64)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("fmt,bs", FORMATS)
@pytest.mark.parametrize("T", [1, 4, 40])
def test_a_nan_or_an_infinity_is_not_lost(T, fmt, bs, dtype):
    """A token with a NaN or an infinity gives NaN, whole; the other tokens' results stay within their bound."""
    print(f"case moe NaN T={T} {fmt} {bs} {dtype}", flush=True)
    r = np.random.default_rng(T + bs)
    weights, v13, v2 = layer(r, 4, 256, 256, fmt, bs)
    for value in (float("nan"), float("inf"), float("-inf")):
        x, logits = inputs(r, T, 256, 4, dtype)
        x[T // 2, 77] = value
        got = q4.moe_q4(x, logits, *weights, 2, fmt=fmt, bs=bs)
        assert got[T // 2].isnan().all()
        keep = [t for t in range(T) if t != T // 2]
        y, e = W.moe(W.as_f64(x)[keep], W.as_f64(logits)[keep], v13, v2, 2, bs, True)
        if dtype == torch.bfloat16:
            e = e + 2.0 ** -8 * (np.abs(y) + e)
        assert (np.abs(W.as_f64(got)[keep] - y) <= e + 1e-30).all()
