"""The paged-cache operators without a GPU: the plain CPU forms against dense or hand-worked ones, and the
entry points' refusals, which happen on the host before any launch."""
import ctypes
import math

import numpy as np
import pytest
import torch

from oracle import paged
from ultra_long_context_b200 import hsa

FAKE = ctypes.c_void_p(1 << 20)   # only ever passed to calls that fail validation first
FAKE2 = ctypes.c_void_p(1 << 21)
ODD2 = ctypes.c_void_p((1 << 20) + 2)
ODD4 = ctypes.c_void_p((1 << 20) + 4)


# ---- the plain forms ----
def test_plan_worked_by_hand():
    table = np.full((4, 3), -1, np.int32)
    table[0, 0], table[2, :2] = 7, (3, 9)
    ring = np.array([5, 4, 8, 1, -1, -1], np.int32)
    # request 0 grows from 60 to 70 (one page), 1 takes a prompt of 65 (two pages), 2 is finished, 3 idles
    cu, slots, total, table2, ring2, pool = paged.page_plan(
        np.array([60, 0, 100, 0]), np.array([10, 65, -1, 0]), table, ring, np.array([0, 4, 0]), 80)
    assert cu.tolist() == [0, 10, 75, 75, 75]
    assert total.tolist() == [70, 65, 0, 0]
    assert slots[:10].tolist() == [7 * 64 + i for i in (60, 61, 62, 63)] + [5 * 64 + i for i in range(6)]
    assert slots[10:75].tolist() == [4 * 64 + i for i in range(64)] + [8 * 64]
    assert slots[75:].tolist() == [-1] * 5
    assert table2[0].tolist() == [7, 5, -1] and table2[1].tolist() == [4, 8, -1]
    assert ring2.tolist() == [5, 4, 8, 1, 3, 9] and pool.tolist() == [3, 6, 0]


def test_plan_refuses_what_does_not_fit():
    table = np.full((5, 2), -1, np.int32)
    table[4, 0] = 6
    ring = np.array([0, 1, 2], np.int32)
    # 0: two of three pages; 1: two more are too many; 2: would fit but comes after; 3: beyond its table;
    # 4: needs no page, so it goes on
    cu, slots, total, table2, _, pool = paged.page_plan(
        np.array([0, 0, 0, 0, 10]), np.array([65, 100, 1, 129, 3]), table, ring, np.array([0, 3, 0]), 1000)
    assert total.tolist() == [65, 0, 0, 0, 13] and pool.tolist() == [2, 3, 3]
    assert (slots[cu[1]:cu[4]] == -1).all() and slots[cu[4]:cu[5]].tolist() == [6 * 64 + i for i in (10, 11, 12)]
    assert (table2[1:4] == -1).all()


def test_prefix_decode_equals_dense_attention():
    rng = np.random.default_rng(5)
    B, H, Hkv, Tq, D, P = 3, 4, 2, 3, 8, 70
    own = np.array([1, 90, -1])       # request 0 has fewer own tokens than query tokens
    Kp, Vp = rng.standard_normal((2, 9, Hkv, 64, D))
    pre, table = np.array([4, 1]), np.array([[0, 2], [7, 3], [-1, -1]])
    q = rng.standard_normal((B, H, Tq, D))
    ref = paged.prefix_decode(q, Kp, Vp, pre, P, table, own, 0.3)
    for b in (0, 1):
        ks = np.concatenate([Kp[pre].transpose(1, 0, 2, 3).reshape(Hkv, -1, D)[:, :P],
                             Kp[table[b]].transpose(1, 0, 2, 3).reshape(Hkv, -1, D)[:, :own[b]]], 1)
        vs = np.concatenate([Vp[pre].transpose(1, 0, 2, 3).reshape(Hkv, -1, D)[:, :P],
                             Vp[table[b]].transpose(1, 0, 2, 3).reshape(Hkv, -1, D)[:, :own[b]]], 1)
        T = P + own[b]
        s = np.einsum("hid,hkd->hik", q[b], np.repeat(ks, 2, 0)) * 0.3
        s[:, np.arange(T)[None] > (T - Tq + np.arange(Tq))[:, None]] = -np.inf
        e = np.exp(s)
        np.testing.assert_allclose(ref["out"][b], np.einsum("hik,hkd->hid", e / e.sum(-1, keepdims=True), np.repeat(vs, 2, 0)),
                                   atol=1e-12)
        np.testing.assert_allclose(ref["lse"][b], np.log(e.sum(-1)), atol=1e-12)
    assert (ref["out"][2] == 0).all() and np.isneginf(ref["lse"][2]).all()


def test_prefix_decode_leaves_out_pages_outside_the_pool():
    rng = np.random.default_rng(6)
    Kp, Vp = rng.standard_normal((2, 4, 1, 64, 8))
    q = rng.standard_normal((1, 1, 1, 8))
    a = paged.prefix_decode(q, Kp, Vp, np.array([2, 4, 1]), 192, np.array([[-1, 0]]), np.array([100]), 0.5)
    b = paged.prefix_decode(q, Kp, Vp, np.array([2, 1]), 128, np.array([[0, 0]]), np.array([36]), 0.5)
    np.testing.assert_allclose(a["out"], b["out"], atol=1e-14)
    assert a["keys"].item() == 164


# ---- refusals of the C entry points ----
def _plan(**kw):
    args = dict(cache_len=FAKE, new_len=FAKE2, B=4, table=FAKE, max_pages=8, ring=FAKE2, num_free=16, pool=FAKE, pool_out=FAKE,
                total=FAKE, cu=FAKE, slots=FAKE2, max_tokens=16, stream=None)
    args.update(kw)
    return hsa.lib().hsa_page_plan(*args.values())


@pytest.mark.parametrize("kw,status", [
    (dict(B=0), -1), (dict(B=8193), -2), (dict(max_pages=0), -1), (dict(max_pages=1 << 30), -2), (dict(num_free=0), -1),
    (dict(num_free=1 << 30), -2), (dict(max_tokens=-1), -1), (dict(cache_len=None), -1), (dict(new_len=None), -1),
    (dict(table=None), -1), (dict(ring=None), -1), (dict(pool=None), -1), (dict(pool_out=None), -1), (dict(total=None), -1),
    (dict(cu=None), -1), (dict(slots=None), -1), (dict(cache_len=ODD4), -1), (dict(new_len=ODD2), -1), (dict(slots=ODD4), -1),
    (dict(ring=FAKE), -1), (dict(slots=FAKE), -1), (dict(cu=FAKE2), -1),
])
def test_plan_rejects_invalid_calls_on_host(kw, status):
    assert _plan(**kw) == status
    assert hsa.hsa_last_error() != ""


def _append(**kw):
    args = dict(K=FAKE, ks=256, V=FAKE, vs=256, slots=FAKE, n=4, Hkv=2, D=128, page=64, Kp=FAKE, Vp=FAKE2, num_pages=8,
                stream=None)
    args.update(kw)
    return hsa.lib().hsa_page_append(*args.values())


@pytest.mark.parametrize("kw,status", [
    (dict(D=96), -2), (dict(page=16), -2), (dict(page=0), -1), (dict(Hkv=0), -1), (dict(num_pages=0), -1), (dict(n=-1), -1),
    (dict(K=None), -1), (dict(V=None), -1), (dict(slots=None), -1), (dict(Kp=None), -1), (dict(Vp=None), -1),
    (dict(K=ODD4), -1), (dict(Vp=ODD4), -1), (dict(slots=ODD4), -1), (dict(ks=260), -1), (dict(vs=248), -1), (dict(Vp=FAKE), -1),
    (dict(num_pages=1 << 30), -2),
])
def test_append_rejects_invalid_calls_on_host(kw, status):
    assert _append(**kw) == status
    assert hsa.hsa_last_error() != ""


def _pre(**kw):
    args = dict(q=FAKE, Kp=FAKE, Vp=FAKE, num_pages=64, ptab=FAKE, mpp=16, plen=FAKE, tab=FAKE, mp=4, own=FAKE, B=4, H=8, Hkv=2,
                Tq=1, D=128, page=64, scale=0.0, out=FAKE, lse=None, ws=FAKE, ws_bytes=1 << 40, stream=None)
    args.update(kw)
    return hsa.lib().hsa_prefix_decode(*args.values())


@pytest.mark.parametrize("kw,status", [
    (dict(D=96), -2), (dict(page=128), -2), (dict(B=0), -1), (dict(B=8193), -2), (dict(H=7), -1), (dict(Hkv=0), -1),
    (dict(Tq=0), -1), (dict(Tq=65), -1), (dict(H=256, Hkv=1, Tq=5), -2), (dict(mpp=-1), -1), (dict(mp=-1), -1),
    (dict(mpp=1 << 25), -2), (dict(mp=1 << 28), -2), (dict(B=64, mp=1 << 24), -2), (dict(num_pages=0), -1), (dict(num_pages=1 << 25), -2), (dict(q=None), -1), (dict(Kp=None), -1),
    (dict(Vp=None), -1), (dict(ptab=None), -1), (dict(plen=None), -1), (dict(tab=None), -1), (dict(own=None), -1),
    (dict(out=None), -1), (dict(q=ODD4), -1), (dict(Kp=ODD4), -1), (dict(out=ODD4), -1), (dict(lse=ODD2), -1), (dict(own=ODD4), -1),
    (dict(ptab=ODD2), -1), (dict(ws=None), -3), (dict(ws_bytes=8), -3), (dict(ws=ODD4), -3), (dict(B=8192, H=2048, Hkv=2048, mp=1), -2),
])
def test_prefix_decode_rejects_invalid_calls_on_host(kw, status):
    assert _pre(**kw) == status
    assert hsa.hsa_last_error() != ""


def test_prefix_decode_workspace_size():
    a = hsa.hsa_prefix_decode_workspace_size(4, 8, 8, 128, 64, 8)
    b = hsa.hsa_prefix_decode_workspace_size(256, 32, 2, 128, 4096, 64)
    assert 0 < a <= b
    assert hsa.hsa_prefix_decode_workspace_size(0, 8, 8, 128, 64, 8) == 0
    assert hsa.hsa_prefix_decode_workspace_size(4, 8, 3, 128, 64, 8) == 0


# ---- the wide kernel's exponential of its own ----
def test_polynomial_exponential_is_as_good_as_its_comment_says():
    """The coefficients as they stand in the source, the kernel's steps in fp32 (a fused multiply-add is one rounding; in fp64 the
    product is exact and the sum nearly so): off by 2^-22 at most, and the clamped ends."""
    import os
    import re

    src = open(os.path.join(os.path.dirname(hsa.__file__), "csrc", "prefix_wide.cu")).read()
    body = src[src.index("pf_exp2_fma(float2 y) {"):]
    coefficients = [np.float32(float.fromhex(a)) for a, b in re.findall(r"\{(0x[0-9a-fp.+-]+)f, (0x[0-9a-fp.+-]+)f\}", body[:body.index("return")]) if a == b]
    assert len(coefficients) == 6

    def exp2(y):
        y = np.clip(y.astype(np.float32), np.float32(-126), np.float32(127))
        t = (y + np.float32(12582912)).astype(np.float32)
        n = (t - np.float32(12582912)).astype(np.float32)
        f = (y.astype(np.float64) - n).astype(np.float32)
        p = np.full_like(f, coefficients[0])
        for c in coefficients[1:]:
            p = (p.astype(np.float64) * f + c).astype(np.float32)
        return (p.view(np.int32) + (t.view(np.int32) << 23)).view(np.float32)

    rng = np.random.default_rng(8)
    y = np.concatenate([rng.uniform(-126, 127, 400000), rng.uniform(-1, 1, 200000), np.arange(-126, 128), np.arange(-126, 127) + 0.5]).astype(np.float32)
    true = np.exp2(y.astype(np.float64))
    assert np.abs(exp2(y) / true - 1).max() <= 2.0**-22
    assert exp2(np.array([-np.inf, -1000.0]))[0] <= 2.0**-126 * 1.000001
    assert (exp2(np.array([128.0, 1e30, np.inf])) >= 2.0**126).all()
