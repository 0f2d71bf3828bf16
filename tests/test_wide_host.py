"""The 8-bit operators without a GPU: exports and headers agree, invalid C calls are refused on the host with the
documented status before any device work, workspace sizes, and pins of the plain 64-bit forms that the GPU tests
compare with (tests/_wide.py)."""
import ctypes
import os
import re

import numpy as np
import pytest
import torch

import block_quantized_bit_amd as q4
from tests import _wide as W

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
OK, NULL, DIM, BLOCK, FORMAT, ALIGN, HIP, RANGE, SCRATCH = range(9)
A = 0x100000  # stands in for a device pointer: every call below fails validation first
LL, P, I = ctypes.c_longlong, ctypes.c_void_p, ctypes.c_int


def declared(header):
    text = open(os.path.join(ROOT, "include", header)).read()
    return sorted(set(re.findall(r"^(?:int|size_t)\s+((?:f8|kv8|moe)_\w+)\(", text, flags=re.M)))


def test_exports_match_the_headers():
    L = q4.lib()
    assert declared("f8.h") == sorted(q4.F8_EXPORTS)
    assert declared("kv8.h") == sorted(q4.KV8_EXPORTS)
    assert declared("moe.h") == sorted(q4.MOE_EXPORTS)
    for name in q4.F8_EXPORTS + q4.KV8_EXPORTS + q4.MOE_EXPORTS:
        assert getattr(L, name) is not None


def func(name, *types, res=I):
    f = ctypes.CDLL(q4.LIB_PATH)[name]
    f.argtypes, f.restype = list(types), res
    return f


def test_f8_refusals():
    rows = func("f8_quantize_rows", I, I, I, P, LL, P, P, P)
    assert rows(4, 128, 1, None, 128, A, A, None) == NULL
    assert rows(4, 128, 2, A, 128, A, A, None) == FORMAT
    assert rows(0, 128, 1, A, 128, A, A, None) == DIM
    assert rows(4, 128, 1, A, 127, A, A, None) == DIM            # rows overlap
    assert rows(4, 1 << 23, 1, A, 1 << 23, A, A, None) == DIM
    assert rows(4, 128, 1, A + 1, 128, A, A, None) == ALIGN
    assert rows(4, 128, 1, A, 128, A + 8, A, None) == ALIGN
    gemm = func("f8_gemm", I, I, I, I, P, P, P, P, P, P)
    assert gemm(4, 128, 8, 0, A, A, A, A, None, None) == NULL
    assert gemm(4, 100, 8, 0, A, A, A, A, A, None) == BLOCK
    assert gemm(4, 128, 8, 7, A, A, A, A, A, None) == FORMAT
    assert gemm(4, 128, 0, 0, A, A, A, A, A, None) == DIM
    assert gemm(1 << 20, 128, 1 << 20, 0, A, A, A, A, A, None) == DIM  # outputs beyond the grid
    assert gemm(4, 128, 8, 0, A, A, A + 4, A, A, None) == ALIGN
    linear = func("f8_linear", I, I, I, I, P, LL, P, P, P, P, P)
    assert linear(4, 128, 8, 0, A, 128, A, A, A, None, None) == NULL
    assert linear(4, 128, 8, 0, A, 128, A, A, A, A + 4, None) == ALIGN
    work = func("f8_linear_work_bytes", I, I, res=ctypes.c_size_t)
    assert work(3, 300) == 3 * 384 + 128 + 256 and work(0, 128) == 0  # codes to 256, three scales a row to 256
    back = func("f8_linear_backward", I, I, I, I, P, LL, P, LL, P, P, P, I, P, P, P)
    ok = [4, 128, 8, 0, A, 8, A, 128, A, A, A, 0, A, A, None]

    def changed(**kw):
        a = list(ok)
        for k, v in kw.items():
            a[int(k[1:])] = v
        return back(*a)
    assert changed(_10=None, _12=None) == NULL                    # no gradient asked for
    assert changed(_8=None) == NULL and changed(_6=None) == NULL and changed(_13=None) == NULL
    assert changed(_11=5) == FORMAT and changed(_3=9) == FORMAT
    assert changed(_5=7) == DIM and changed(_12=A + 2) == ALIGN


class Cache(ctypes.Structure):
    _fields_ = [(n, I) for n in ("format", "pages", "kv_heads", "page_size", "head_dim", "batch", "max_pages")] + \
               [(n, P) for n in ("k_codes", "v_codes", "k_scale", "v_scale", "page_table", "kv_len", "cu")]


def cache(**kw):
    c = Cache(0, 10, 2, 16, 64, 3, 4, A, A, A, A, A, A, A)
    for k, v in kw.items():
        setattr(c, k, v)
    return ctypes.byref(c)


@pytest.mark.parametrize("kw,status", [
    (dict(format=2), FORMAT), (dict(page_size=24), BLOCK), (dict(page_size=8), BLOCK), (dict(page_size=512), BLOCK),
    (dict(head_dim=96), DIM), (dict(pages=0), DIM), (dict(batch=0), DIM), (dict(batch=40000), DIM),
    (dict(max_pages=1 << 28), DIM), (dict(k_codes=None), NULL), (dict(cu=None), NULL), (dict(v_codes=A + 8), ALIGN),
    (dict(kv_len=A + 2), ALIGN),
])
def test_kv8_cache_refusals(kw, status):
    app = func("kv8_append", P, I, I, I, P, LL, P, LL, P)
    read = func("kv8_read", P, I, I, I, P, P, P)
    attend = func("kv8_attention", P, I, I, I, I, I, P, LL, ctypes.c_float, I, P, P, P, P)
    assert app(cache(**kw), 3, 1, 0, A, 128, A, 128, None) == status
    assert read(cache(**kw), 3, 1, 0, A, A, None) == status
    assert attend(cache(**kw), 3, 1, 64, 4, 0, A, 256, 1.0, 0, A, None, A, None) == status


def test_kv8_call_refusals():
    app = func("kv8_append", P, I, I, I, P, LL, P, LL, P)
    assert app(None, 3, 1, 0, A, 128, A, 128, None) == NULL
    assert app(cache(), 3, 1, 0, None, 128, A, 128, None) == NULL
    assert app(cache(), 3, 1, 5, A, 128, A, 128, None) == FORMAT
    assert app(cache(), 0, 1, 0, A, 128, A, 128, None) == DIM
    assert app(cache(), 3, 0, 0, A, 128, A, 128, None) == DIM
    assert app(cache(), 3, 1, 0, A, 127, A, 128, None) == DIM
    assert app(cache(), 3, 1, 0, A + 2, 128, A, 128, None) == ALIGN
    attend = func("kv8_attention", P, I, I, I, I, I, P, LL, ctypes.c_float, I, P, P, P, P)

    def call(total=3, new=1, kv=64, heads=4, dt=0, q=A, stride=256, scale=1.0, window=0, out=A, lse=None, work=A):
        return attend(cache(), total, new, kv, heads, dt, q, stride, scale, window, out, lse, work, None)
    assert call(heads=3) == DIM and call(heads=0) == DIM and call(kv=0) == DIM and call(window=-1) == DIM
    assert call(stride=255) == DIM and call(q=None) == NULL and call(work=None) == NULL and call(out=A + 8) == ALIGN
    assert call(scale=float("nan")) == RANGE and call(scale=float("inf")) == RANGE and call(lse=A + 1) == ALIGN
    size = func("kv8_attention_work_bytes", P, I, I, I, I, res=ctypes.c_size_t)
    assert size(cache(), 3, 1, 64, 3) == 0
    assert 0 < size(cache(), 3, 1, 64, 4) <= size(cache(max_pages=4096), 3, 1, 65536, 4)


def test_moe_refusals():
    f = func("moe_q4", *[I] * 8, *[P] * 8, I, P, P, P)

    def call(T=2, H=128, inter=128, E=4, k=2, bs=32, fmt=0, dt=0, x=A, b=None, w2=A, out=A, work=A):
        return f(T, H, inter, E, k, bs, fmt, dt, x, A, A, A, b, w2, A, b, 1, out, work, None)
    assert call(fmt=2) == FORMAT and call(dt=3) == FORMAT
    assert call(bs=64) == BLOCK and call(fmt=1, bs=32, b=A) == BLOCK and call(H=100) == BLOCK
    assert call(T=0) == DIM and call(T=65) == DIM and call(E=513) == DIM and call(k=5) == DIM and call(k=0) == DIM
    assert call(E=64, k=17) == DIM and call(H=65536) == DIM
    assert call(fmt=1, bs=64) == NULL and call(x=None) == NULL and call(work=None) == NULL
    assert call(w2=A + 8) == ALIGN and call(out=A + 4) == ALIGN
    size = func("moe_q4_work_bytes", *[I] * 6, res=ctypes.c_size_t)
    assert size(2, 128, 128, 4, 5, 32) == 0 and size(2, 128, 128, 4, 2, 32) > 4 * 128


def test_binding_refuses_host_tensors():
    if torch.cuda.is_available():
        pytest.skip("host-only check")
    with pytest.raises(ValueError):
        q4.f8_linear(torch.zeros(2, 128), torch.zeros(4, 128).to(W.F8), torch.zeros(1, 1))
    with pytest.raises(TypeError):
        q4.f8_linear([1.0], None, None)
    with pytest.raises(ValueError):
        q4.moe_q4(torch.zeros(1, 64), torch.zeros(1, 2), *[torch.zeros(1)] * 6, 1)


# ---- the plain forms --------------------------------------------------------------------

def test_e4m3_is_torchs():
    grid = torch.arange(256, dtype=torch.uint8).view(W.F8).float()
    grid = grid[torch.isfinite(grid)].unique()
    mid = (grid[:-1] + grid[1:]) / 2
    r = torch.from_numpy(np.random.default_rng(0).uniform(-448, 448, 50000).astype(np.float32))
    small = r * 2.0 ** -14
    for x in (grid, mid, torch.nextafter(mid, torch.tensor(0.0)), r, small):
        assert np.array_equal(W.e4m3(x.double().numpy()), x.to(W.F8).double().numpy())


def test_products_are_plain_matrix_products():
    r = np.random.default_rng(1)
    x, w = r.standard_normal((5, 300)), r.standard_normal((140, 300))
    xc, xs = W.f8_rows(x.astype(np.float32))
    wc, ws = W.f8_weights(w.astype(np.float32))
    xv = xc * np.repeat(xs.T, 128, 1)
    wv = wc * np.repeat(np.repeat(ws, 128, 0)[:140], 128, 1)
    y, a = W.f8_product(xc, xs, wc, ws)
    assert np.allclose(y, xv @ wv.T, rtol=1e-12) and (a >= np.abs(y) * (1 - 1e-12)).all()
    assert np.abs(xv[:, :300] - x).max() <= np.abs(x).max() / 16 + 1e-6   # three fraction bits
    wc2, ws2 = W.f8_rows(w.astype(np.float32))
    y, _ = W.f8_product_rows(xc, xs, wc2, ws2)
    assert np.allclose(y, xv @ (wc2 * np.repeat(ws2.T, 128, 1)).T, rtol=1e-12)


@pytest.mark.parametrize("kind", [torch.int8, W.F8])
def test_plain_cache(kind):
    r = np.random.default_rng(2)
    c = W.PlainCache(3, 1, 16, 8, kind)
    kv = r.standard_normal((2, 20, 1, 8)).astype(np.float32).astype(np.float64)
    c.append(kv[:, :10], [2, 0], 0)
    first = c.scale[0, 2, 0]
    c.append(4 * kv[:, 10:], [2, 0], 10)
    assert c.scale[0, 2, 0] > first and c.scale[0, 1, 0] == 0
    got = c.values(0, [2, 0], 0, 20)
    want = np.concatenate([kv[0, :10], 4 * kv[0, 10:]])
    step = np.repeat(c.scale[0, [2, 0], 0], 16)[:20, None, None] * (1.5 if kind == torch.int8 else 40)
    assert (np.abs(got - want) <= step).all()
    assert (c.values(0, [2, 0], -2, 1)[:2] == 0).all()


def test_plain_attention_is_torchs():
    r = np.random.default_rng(3)
    q, k, v = r.standard_normal((6, 4, 8)), r.standard_normal((9, 2, 8)), r.standard_normal((9, 2, 8))
    place = 3 + np.arange(6)
    for window in (0, 4):
        out, lse, _ = W.attention(q, k, v, place, 0.3, window)
        t = np.arange(9)
        see = (t <= place[:, None]) & ((t > place[:, None] - window) if window else True)
        kt, vt = (torch.from_numpy(np.repeat(a, 2, 1)).transpose(0, 1) for a in (k, v))
        s = (torch.from_numpy(q).transpose(0, 1) @ kt.transpose(1, 2) * 0.3).masked_fill(~torch.from_numpy(see), -torch.inf)
        assert np.allclose(out, (s.softmax(-1) @ vt).transpose(0, 1).numpy(), rtol=1e-12)
        assert np.allclose(lse, s.logsumexp(-1).T.numpy(), rtol=1e-12)
    out, lse, _ = W.attention(q[:1], k, v, np.array([-1]), 0.3, 0)
    assert (out == 0).all() and (lse == -np.inf).all()


def test_plain_routing():
    l = np.array([1.0, 3.0, 3.0, -np.inf, np.nan, 2.0])
    got = W.route(l, 3, True)
    assert [e for e, _ in got] == [1, 2, 5] and abs(sum(w for _, w in got) - 1) < 1e-12
    full = np.exp([1.0, 3.0, 3.0, 2.0])
    assert np.allclose([w for _, w in W.route(l, 2, False)], np.exp(3.0) / full.sum())
    assert W.route(np.full(4, -np.inf), 2, True) == []
    assert len(W.route(l, 6, True)) == 4


@pytest.mark.parametrize("mistake", ["no causal mask", "scale of another page", "mean in place of sum"])
def test_a_planted_mistake_exceeds_the_bounds(mistake):
    """The bounds of the attention tests are far below what a plausible mistake in the formula gives."""
    from tests.test_kv8 import bound
    r = np.random.default_rng(4)
    q, k, v = r.standard_normal((4, 2, 16)), r.standard_normal((40, 1, 16)), r.standard_normal((40, 1, 16))
    want, _, mass = W.attention(q, k, v, 36 + np.arange(4), 0.25, 0)
    if mistake == "no causal mask":
        got, _, _ = W.attention(q, k, v, np.full(4, 39), 0.25, 0)
    elif mistake == "scale of another page":
        got, _, _ = W.attention(q, k, np.where(np.arange(40)[:, None, None] < 16, 1.1 * v, v), 36 + np.arange(4), 0.25, 0)
    else:
        got = want / np.arange(37, 41)[:, None, None]
    spread = 0.25 * max((np.abs(q[:, h]) @ np.abs(k[:, 0]).T).max() for h in range(2))
    assert (np.abs(got - want) > bound(mass, 40, spread, torch.bfloat16)).any()


def test_sizes_are_refused_as_such_without_a_workspace():
    """Sizes beyond the limits have no workspace (its size is 0, its pointer may be null): the status names the size."""
    linear = func("f8_linear", I, I, I, I, P, LL, P, P, P, P, P)
    back = func("f8_linear_backward", I, I, I, I, P, LL, P, LL, P, P, P, I, P, P, P)
    big = 1 << 23
    for M, K, N in ((big, 128, 8), (4, big, 8), (4, 128, big), (0, 128, 8)):
        assert linear(M, K, N, 0, A, K, A, A, A, None, None) == DIM
        assert back(M, K, N, 0, A, N, A, K, A, A, A, 0, A, None, None) == DIM
    assert linear(1 << 21, 128, 1 << 21, 0, A, 128, A, A, A, None, None) == DIM  # outputs beyond the grid
    assert back(4, 128, 8, 0, A, 8, A, 128, A, A, A, 0, A, None, None) == NULL
    assert linear(4, 128, 8, 0, None, 128, A, A, A, None, None) == NULL
