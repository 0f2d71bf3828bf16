"""The e4m3 block-128 product and its gradients on the GPU against 64-bit values on the CPU.

Codes and scales have to be the defined ones exactly; products stay within the bound of float32 sums
(tests/_wide.py, f8_bound), derived from the number of additions."""
import numpy as np
import pytest
import torch

import block_quantized_bit_amd as q4
from tests import _wide as W

pytestmark = pytest.mark.gpu

DTYPES = [torch.bfloat16, torch.float32]


def activations(M, K, dtype, seed=0):
    r = np.random.default_rng(seed + 131 * M + K)
    x = r.standard_normal((M, K)) * np.where(r.random(K) < 0.02, 16.0, 1.0)
    return torch.from_numpy(x.astype(np.float32)).cuda().to(dtype)


def weights(N, K, seed=0):
    """(codes tensor, scales tensor, code values, scales) of random weights, quantized by the plain form."""
    r = np.random.default_rng(seed + 7 * N + K)
    c, s = W.f8_weights((0.02 * r.standard_normal((N, K))).astype(np.float32))
    return W.to_f8(c), W.gpu32(s), c, s


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("M,K", [(1, 1), (1, 128), (3, 127), (5, 129), (17, 640), (2, 1000), (130, 256), (64, 4096)])
def test_quantize_rows_exact(M, K, dtype):
    print(f"case quantize_rows {M} {K} {dtype}", flush=True)
    x = activations(M, K, dtype)
    c, s = W.f8_rows(W.as_f64(x))
    xq, xs = q4.f8_quantize_act(x)
    assert np.array_equal(W.as_f64(xq), c) and np.array_equal(W.as_f64(xs), s)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("M,K", [(1, 1), (128, 64), (127, 65), (300, 100), (129, 256)])
def test_quantize_cols_exact(M, K, dtype):
    print(f"case quantize_cols {M} {K} {dtype}", flush=True)
    x = activations(M, K, dtype)
    c, s = W.f8_rows(W.as_f64(x).T)
    xt, xts = q4.f8_quantize_act_t(x)
    assert np.array_equal(W.as_f64(xt), c) and np.array_equal(W.as_f64(xts), s)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("N,K", [(1, 1), (128, 128), (200, 300), (129, 127)])
def test_quantize_weights_and_transpose_exact(N, K, dtype):
    print(f"case quantize_weights {N} {K} {dtype}", flush=True)
    w = (0.02 * activations(N, K, torch.float32)).to(dtype)
    c, s = W.f8_weights(W.as_f64(w))
    wq, ws = q4.f8_quantize_weights(w)
    assert np.array_equal(W.as_f64(wq), c) and np.array_equal(W.as_f64(ws), s)
    wqt, wst = q4.f8_transpose_weights(wq, ws, K)
    ct = W.pad128(c, 0)[:, :K].T
    assert np.array_equal(W.as_f64(wqt), ct) and np.array_equal(W.as_f64(wst), s.T)


def test_quantizer_ties_subnormals_and_extremes():
    # amax 448 makes the scale 1: the values themselves are rounded. Ties between neighbours, the subnormal
    # range (steps of 2^-9), a block of zeros, a block whose scale is subnormal, and one at the top of float32.
    x = np.zeros((4, 256), dtype=np.float32)
    grid = np.unique(np.abs(W.e4m3(np.linspace(0, 448, 20000))))
    mid = (grid[:-1] + grid[1:]) / 2
    x[0, :len(mid[:127])] = mid[:127]
    x[0, 127] = 448
    x[1, :len(mid[-100:])] = -mid[-100:]
    x[1, 127] = -448
    x[1, 128:] = np.arange(128) * 2.0 ** -10
    x[1, 255] = 448
    x[2, :128] = np.arange(128) * 2.0 ** -149
    x[3, :128] = np.float32(3e38) * np.linspace(-1, 1, 128).astype(np.float32)
    c, s = W.f8_rows(x.astype(np.float64))
    xq, xs = q4.f8_quantize_act(torch.from_numpy(x).cuda())
    assert np.array_equal(W.as_f64(xs), s) and np.array_equal(W.as_f64(xq), c)


def test_nan_and_infinity_stay_in_their_place():
    x = activations(3, 256, torch.float32)
    x[0, 5] = float("nan")
    x[1, 200] = float("inf")
    clean = x.clone()
    clean[0, 5] = 0.0
    xq, xs = q4.f8_quantize_act(x)
    c, s = W.f8_rows(W.as_f64(clean))
    got = W.as_f64(xq)
    assert np.isnan(got[0, 5])
    got[0, 5] = 0.0
    assert np.array_equal(got[0], c[0]) and np.array_equal(got[2], c[2])
    assert np.isinf(W.as_f64(xs)[1, 1])
    wq, ws, _, _ = weights(48, 256)
    y = W.as_f64(q4.f8_linear(x, wq, ws))
    assert np.isnan(y[0]).all() and np.isnan(y[1]).all() and np.isfinite(y[2]).all()


SHAPES = [(1, 1, 1), (1, 128, 16), (1, 4096, 257), (2, 136, 40), (4, 1000, 33), (5, 127, 130), (16, 384, 128),
          (17, 256, 100), (33, 640, 65), (64, 4096, 96), (65, 256, 130), (128, 128, 128), (200, 384, 1536),
          (130, 300, 515), (1000, 256, 129)]


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("M,K,N", SHAPES)
def test_linear(M, K, N, dtype):
    print(f"case linear {M} {K} {N} {dtype}", flush=True)
    x = activations(M, K, dtype)
    wq, ws, c, s = weights(N, K)
    y, a = W.f8_product(*W.f8_rows(W.as_f64(x)), c, s)
    out = torch.full((M, N), float("nan"), dtype=dtype, device="cuda")
    got = W.as_f64(q4.f8_linear(x, wq, ws, out=out))
    assert (np.abs(got - y) <= W.f8_bound(a, (K + 127) // 128, y, dtype)).all()
    # the product of ready codes is the same computation
    xq, xs = q4.f8_quantize_act(x)
    two = q4.f8_gemm(xq, xs, wq, ws, dtype=dtype)
    assert (np.abs(W.as_f64(two) - y) <= W.f8_bound(a, (K + 127) // 128, y, dtype)).all()


@pytest.mark.parametrize("M", [3, 70, 2100])
def test_linear_large_tiles_and_strided_rows(M):
    # 2100 x 8448: enough tiles for the large ones; x is a slice of a wider tensor whose rows start off 16 bytes
    K, N = 256, 8448 if M > 1000 else 300
    print(f"case linear strided {M}", flush=True)
    wide = activations(M, K + 37, torch.bfloat16)
    x = wide[:, 5:5 + K]
    wq, ws, c, s = weights(N, K)
    y, a = W.f8_product(*W.f8_rows(W.as_f64(x)), c, s)
    got = W.as_f64(q4.f8_linear(x, wq, ws))
    assert (np.abs(got - y) <= W.f8_bound(a, 2, y, torch.bfloat16)).all()


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("M,K,N", [(1, 128, 128), (1, 1, 1), (100, 130, 50), (128, 256, 384), (515, 300, 200),
                                   (300, 127, 129)])
def test_backward(M, K, N, dtype):
    print(f"case backward {M} {K} {N} {dtype}", flush=True)
    x = activations(M, K, dtype)
    dy = (0.01 * activations(M, N, torch.float32, 1)).to(dtype)
    wq, ws, c, s = weights(N, K)
    wqt, wst = q4.f8_transpose_weights(wq, ws, K)
    dx, dw = q4.f8_linear_backward(dy, x, wqt, wst)
    xf, dyf = W.as_f64(x), W.as_f64(dy)
    ct = W.pad128(c, 0)[:, :K].T
    y, a = W.f8_product(*W.f8_rows(dyf), ct, s.T)
    assert (np.abs(W.as_f64(dx) - y) <= W.f8_bound(a, (N + 127) // 128, y, dtype)).all()
    y, a = W.f8_product_rows(*W.f8_rows(dyf.T), *W.f8_rows(xf.T))
    assert dw.dtype == dtype
    assert (np.abs(W.as_f64(dw) - y) <= W.f8_bound(a, (M + 127) // 128, y, dtype)).all()
    exact = torch.full((N, K), float("nan"), dtype=torch.float32, device="cuda")
    q4.f8_linear_backward(dy, x, wqt, wst, need_dx=False, dw=exact)
    assert (np.abs(W.as_f64(exact) - y) <= W.f8_bound(a, (M + 127) // 128, y, torch.float32)).all()
    only_dx = q4.f8_linear_backward(dy, None, wqt, wst, need_dw=False)
    only_dw = q4.f8_linear_backward(dy, x, None, None, need_dx=False)
    assert only_dx[1] is None and torch.equal(only_dx[0], dx)
    assert only_dw[0] is None and torch.equal(only_dw[1], dw)


def test_gradient_against_differences():
    """Where the inputs are e4m3 values under scale 1, the quantizers change nothing: the loss sum(dy * y) is linear
    in x and in w, so a difference quotient of any step is the gradient up to float32 sums."""
    M, K, N = 140, 130, 70
    r = np.random.default_rng(5)

    def grid(*shape):
        v = W.e4m3(r.uniform(-8, 8, shape))
        v[..., 0] = 448.0  # pins a block's scale at 1
        v[:, 128:129] = 448.0
        return v

    x, w = grid(M, K), W.e4m3(r.uniform(-8, 8, (N, K)))
    w[0, 0], w[0, 128] = 448.0, 448.0
    dy = W.e4m3(r.uniform(-8, 8, (M, N)))
    dy[:, 0] = 448.0   # blocks along N
    dy[0], dy[128] = 448.0, 448.0  # and along the tokens
    x[0], x[128] = 448.0, 448.0
    wq, ws = q4.f8_quantize_weights(gpu32(w))
    assert np.array_equal(W.as_f64(wq)[:, :K], w) and (W.as_f64(ws) == 1).all()
    wqt, wst = q4.f8_transpose_weights(wq, ws, K)
    dx, dw = q4.f8_linear_backward(gpu32(dy), gpu32(x), wqt, wst)
    scale = np.abs(dy).sum() * 448 * 448 * 2.0 ** -23

    def loss(xv, wv):
        q, s = q4.f8_quantize_weights(gpu32(wv))
        return float((W.as_f64(q4.f8_linear(gpu32(xv), q, s)) * dy).sum())

    base = loss(x, w)
    for m, k in [(1, 1), (77, 64), (139, 129), (129, 3)]:
        step = x.copy()
        step[m, k] = 256.0
        assert abs((loss(step, w) - base) / (256.0 - x[m, k]) - W.as_f64(dx)[m, k]) <= scale
    for n, k in [(1, 1), (69, 64), (33, 129)]:
        step = w.copy()
        step[n, k] = 256.0
        assert abs((loss(x, step) - base) / (256.0 - w[n, k]) - W.as_f64(dw)[n, k]) <= scale


gpu32 = W.gpu32


def test_calls_are_repeatable_and_follow_the_stream():
    x = activations(300, 512, torch.bfloat16)
    wq, ws, _, _ = weights(200, 512)
    first = q4.f8_linear(x, wq, ws)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        again = q4.f8_linear(x, wq, ws)
    given = q4.f8_linear(x, wq, ws, stream=side)
    side.synchronize()
    assert torch.equal(first, again) and torch.equal(first, given)


def test_refusals():
    x = activations(4, 256, torch.float32)
    wq, ws, _, _ = weights(64, 256)
    with pytest.raises(ValueError):
        q4.f8_linear(x.half(), wq, ws)
    with pytest.raises(ValueError):
        q4.f8_linear(x.cpu(), wq, ws)
    with pytest.raises(ValueError):
        q4.f8_linear(x[:, :100], wq, ws)      # weights of another K
    with pytest.raises(ValueError):
        q4.f8_linear(x.t(), wq, ws)           # columns, not rows, are contiguous
    with pytest.raises(ValueError):
        q4.f8_linear(x, wq.view(torch.uint8), ws)
    with pytest.raises(ValueError):
        q4.f8_linear(x, wq, ws[:, :1])
    with pytest.raises(ValueError):
        q4.f8_linear(x, wq, ws, work=torch.empty(8, dtype=torch.uint8, device="cuda"))
    with pytest.raises(ValueError):
        q4.f8_linear(x[:0], wq, ws)
    with pytest.raises(ValueError):
        q4.f8_linear_backward(x, x[:2], wq, ws)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("K", [100, 300, 640, 1152])
def test_linear_middle_tiles(K, dtype):
    """288 tiles of 128 x 128 (fewer than 256 of 256 x 256), ragged on all sides: one block of k, and numbers of blocks
    that are no multiple of the four stages."""
    M, N = 1030, 3970
    print(f"case linear middle tiles {M} {K} {N} {dtype}", flush=True)
    x = activations(M, K, dtype)
    wq, ws, c, s = weights(N, K)
    y, a = W.f8_product(*W.f8_rows(W.as_f64(x)), c, s)
    out = torch.full((M, N), float("nan"), dtype=dtype, device="cuda")
    got = W.as_f64(q4.f8_linear(x, wq, ws, out=out))
    assert (np.abs(got - y) <= W.f8_bound(a, (K + 127) // 128, y, dtype)).all()


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("M,K,N", [(70, 1030, 3970), (700, 1030, 3970), (300, 4100, 4100)])
def test_weight_gradient_middle_and_large_tiles(M, K, N, dtype):
    """288 tiles of 128 x 128, and for bfloat16 289 of 256 x 256, with scales per row on both sides; M gives one, three
    and six blocks."""
    print(f"case weight gradient tiles {M} {K} {N} {dtype}", flush=True)
    x = activations(M, K, dtype)
    dy = (0.01 * activations(M, N, torch.float32, 1)).to(dtype)
    dw = torch.full((N, K), float("nan"), dtype=dtype, device="cuda")
    q4.f8_linear_backward(dy, x, None, None, need_dx=False, dw=dw)
    y, a = W.f8_product_rows(*W.f8_rows(W.as_f64(dy).T), *W.f8_rows(W.as_f64(x).T))
    assert (np.abs(W.as_f64(dw) - y) <= W.f8_bound(a, (M + 127) // 128, y, dtype)).all()


def test_flags_without_a_truth_value():
    """need_dx and need_dw are asked for their truth; an object that has none raises its own error."""
    x, dy = activations(4, 128, torch.float32), activations(4, 64, torch.float32)
    with pytest.raises(RuntimeError, match="[Bb]oolean"):
        q4.f8_linear_backward(dy, x, None, None, need_dx=False, need_dw=torch.ones(2))
