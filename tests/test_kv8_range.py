"""Attention over the 8-bit cache where weights lie many powers of two below the largest, and with value scales from
2^-100 up, in the kernels for few and for many rows, against 64-bit values on the CPU."""
import numpy as np
import pytest
import torch

import block_quantized_bit_amd as q4
from tests import _wide as W

pytestmark = pytest.mark.gpu

DTYPES = [torch.bfloat16, torch.float32]
KINDS = [torch.int8, torch.float8_e4m3fn]


def i32(values):
    return torch.tensor(values, dtype=torch.int32, device="cuda")


def random_cache(r, L, P, d, kind):
    """One sequence of L tokens, one head, codes over a quarter of their range, pages in random order."""
    pages = (L + P - 1) // P
    cache = W.PlainCache(pages, 1, P, d, kind)
    top = W.kv_top(kind)
    cache.codes[:] = W.kv_round(np.clip(r.standard_normal(cache.codes.shape) * top / 4, -top, top), kind)
    cache.scale[:] = (r.uniform(0.5, 1.5, cache.scale.shape) * 3 / top).astype(np.float32)
    return cache, r.permutation(pages)


def bound(mass, keys, spread, flush, dtype):
    """Distance allowed between a result and the 64-bit one, from sum p|v| (mass). Scores: as queries are two f16
    halves and the sums of their products float32, 2^-20 of sum |q k| (spread), four times for the exponential, its
    factors and the reference. Sums: every float32 addition and every factor loses at most 2^-24, and a sum takes one
    addition for 32 keys in a matrix instruction, one for 64 between chunks and one for each join or change of the
    reference. float32 results have float32 weights. bfloat16 ones have weights of one f16 (2^-11 of themselves, or
    2^-25 below f16's smallest normal number, which adds up to `flush`), and are rounded by 2^-8."""
    e = mass * (4 * 2.0 ** -20 * spread + (keys / 16 + 64) * 2.0 ** -24)
    if dtype == torch.bfloat16:
        e = e + mass * (2.0 ** -11 + 2.0 ** -8 * 1.01) + 1.01 * flush
    return e


def check(q, cache, table, L, dtype, scale):
    n, heads, d = q.shape
    lse = torch.full((n, heads), float("nan"), device="cuda")
    out = q4.kv8_attention(q, *cache.tensors(), i32(table[None].tolist()), i32([L]), i32([0, n]), n, L, scale=scale,
                           lse=lse)
    k, v = (cache.values(w, table, 0, L) for w in range(2))
    qf, place = W.as_f64(q), L - n + np.arange(n)
    want, wlse, mass = W.attention(qf, k, v, place, scale, 0)
    spread = scale * max((np.abs(qf[:, h]) @ np.abs(k[:, 0]).T).max() for h in range(heads))
    # the largest weight is held at 2^11 at least (at the clamped scale): see the kernels' reference
    flush = L * 2.0 ** -36 * W.kv_top(cache.kind) * max(cache.scale[1].max(), 2.0 ** -80)
    err, allowed = np.abs(W.as_f64(out) - want), bound(mass, L, spread, flush, dtype)
    print(f"largest part of the bound {(err / allowed).max():.3g}, relative error "
          f"{np.sqrt((err ** 2).sum() / (want ** 2).sum()):.3g}", flush=True)
    assert (err <= allowed).all()
    # the errors of weights do not depend on the values: the result's relative root mean square is one weight's error
    # beside the rounding of the result (bfloat16: 2^-9 at worst each, here 2^-8), or beside that of the scores
    rms = np.sqrt((err ** 2).sum() / (want ** 2).sum())
    assert rms <= (2.0 ** -8 if dtype == torch.bfloat16 else 2.0 ** -20 * (spread + 1))
    assert (np.abs(W.as_f64(lse) - wlse) <= 4 * 2.0 ** -20 * (spread + 1) + (L / 16 + 64) * 2.0 ** -24).all()


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("n", [1, 130])
@pytest.mark.parametrize("share", [0.7, 0.99, 0.9999])
def test_a_token_of_no_value_takes_most_of_the_weight(share, n, dtype, kind):
    """The first token has `share` of the weight and zero values, so that the result is the other 8191 tokens' alone,
    each of whose weights is 2^-14 to 2^-27 of the largest."""
    print(f"case share {share} n={n} {dtype} {kind}", flush=True)
    r = np.random.default_rng(int(share * 1e4) + n)
    L, P, d, heads = 8192, 64, 64, 4
    cache, table = random_cache(r, L, P, d, kind)
    cache.codes[0, :, :, :, 0] = 0  # the first value of a key tells the first token from the others
    first = cache.codes[:, table[0], 0, 0]
    first[0], first[0, 0], first[1] = 0.0, 64.0, 0.0
    q = W.as_f64((0.5 * torch.from_numpy(r.standard_normal((n, heads, d)))).to(dtype))
    k = cache.values(0, table, 0, L)[:, 0]
    scale = d ** -0.5
    for i in range(n):
        see = slice(1, L - n + i + 1)
        s = scale * (q[i] @ k[see].T)
        others = s.max(1) + np.log(np.exp(s - s.max(1, keepdims=True)).sum(1))
        q[i, :, 0] = (others + np.log(share / (1 - share))) / (scale * k[0, 0])
    check(torch.from_numpy(q.astype(np.float32)).cuda().to(dtype), cache, table, L, dtype, scale)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("n", [1, 100])
@pytest.mark.parametrize("low,high", [(-100, -84), (-100, 20), (-40, 20)])
def test_value_scales_of_any_size(low, high, n, dtype):
    print(f"case scales 2^{low} .. 2^{high} n={n} {dtype}", flush=True)
    r = np.random.default_rng(n - low)
    cache, table = random_cache(r, 200, 16, 64, torch.int8)
    cache.scale[1] = 2.0 ** r.integers(low, high, cache.scale[1].shape)
    cache.scale[1, table[3]] = 0.0
    cache.codes[1, table[3]] = 0.0
    q = torch.from_numpy(r.standard_normal((n, 4, 64)).astype(np.float32)).cuda().to(dtype)
    check(q, cache, table, 200, dtype, 0.125)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("n,L", [(1, 40), (1, 3000), (100, 150), (100, 3000)])
def test_a_query_with_a_nan(n, L, dtype):
    """One head's last query holds a NaN: its result and its lse are NaN (not those of a query that sees no key), every
    other one is as it was. Few and many rows, in one part and in splits."""
    print(f"case NaN query n={n} L={L} {dtype}", flush=True)
    r = np.random.default_rng(n + L)
    cache, table = random_cache(r, L, 64, 64, torch.int8)
    q = torch.from_numpy(r.standard_normal((n, 4, 64)).astype(np.float32)).cuda().to(dtype)
    q[-1, 2, 7] = float("nan")
    lse = torch.zeros(n, 4, device="cuda")
    out = q4.kv8_attention(q, *cache.tensors(), i32(table[None].tolist()), i32([L]), i32([0, n]), n, L, lse=lse)
    assert out[-1, 2].isnan().all() and lse[-1, 2].isnan()
    k, v = (cache.values(w, table, 0, L) for w in range(2))
    qf = W.as_f64(q)
    qf[-1, 2] = 0.0
    want, wlse, mass = W.attention(qf, k, v, L - n + np.arange(n), 0.125, 0)
    spread = 0.125 * max((np.abs(qf[:, h]) @ np.abs(k[:, 0]).T).max() for h in range(4))
    good = np.ones((n, 4), dtype=bool)
    good[-1, 2] = False
    flush = L * 2.0 ** -36 * 127 * cache.scale[1].max()
    assert (np.abs(W.as_f64(out) - want) <= bound(mass, L, spread, flush, dtype))[good].all()
    assert (np.abs(W.as_f64(lse) - wlse)[good] <= 4 * 2.0 ** -20 * (spread + 1) + (L / 16 + 64) * 2.0 ** -24).all()


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("window", [2 ** 31 - 1, 2 ** 30, 2 ** 30 - 1])
@pytest.mark.parametrize("L,n", [(40, 1), (3, 6), (90, 100), (300, 100)])
def test_a_window_as_long_as_an_int_can_say(L, n, window, dtype):
    """Such a window hides nothing, also where queries stand before position 0 (more of them than the length)."""
    print(f"case window {window} L={L} n={n} {dtype}", flush=True)
    r = np.random.default_rng(L + n)
    cache, table = random_cache(r, L, 16, 64, torch.int8)
    q = torch.from_numpy(r.standard_normal((n, 4, 64)).astype(np.float32)).cuda().to(dtype)
    args = (*cache.tensors(), i32(table[None].tolist()), i32([L]), i32([0, n]), n, L)
    want = q4.kv8_attention(q, *args)
    assert n > L or want.abs().amin() > 0
    assert torch.equal(q4.kv8_attention(q, *args, window=window), want)
