"""Refusals of the attention and cache entry points, on the host before anything touches CUDA (the pointers are never
dereferenced), and the host page tables of the oracle."""
from __future__ import annotations

import ctypes
import math
import os
import subprocess
import sys

import numpy as np
import pytest
import torch

from oracle import attention as A
from ternary_weight_linear_int8_b200 import bitnet as B

P = [0x10000000 * (i + 1) for i in range(14)]      # far apart, 16-byte aligned
OK_KV = dict(table=P[10], lens=P[11], refs=P[12], n_slots=4, max_pages=8, n_pages=32, page_size=16)


@pytest.fixture(scope="module")
def L():
    return B.lib()


def kv(**kw):
    return ctypes.byref(B.KvTables(*[dict(OK_KV, **kw)[f] for f, _ in B.KvTables._fields_]))


BAD_KV = [(dict(table=None), 1), (dict(lens=None), 1), (dict(refs=None), 1), (dict(n_slots=0), 2), (dict(n_slots=65537), 2),
          (dict(max_pages=0), 2), (dict(n_pages=0), 2), (dict(page_size=0), 2), (dict(page_size=24), 2),
          (dict(page_size=1040), 2), (dict(max_pages=1 << 28), 2), (dict(table=P[10] + 2), 3), (dict(lens=P[11] + 1), 3)]


def test_prompt_refusals(L):
    def call(**kw):
        a = dict(q=P[0], qs=2560, k=P[1], ks=512, v=P[2], vs=512, cq=P[3], ck=P[4], B=3, Tq=100, Tk=90, Hq=20, Hkv=4,
                 D=128, scale=0.1, y=P[5], ys=2560, lse=None)
        a.update(kw)
        return L.bitnet_attn_prompt(*a.values(), None)

    for name in ("q", "k", "v", "cq", "ck", "y"):
        assert call(**{name: None}) == 1
    for s in (0.0, -1.0, math.nan, math.inf):
        assert call(scale=s) == 1
    for kw in (dict(B=0), dict(Tq=0), dict(Tk=0), dict(Tq=1 << 31), dict(Hq=19), dict(Hkv=0), dict(Hkv=3), dict(D=96),
               dict(D=256), dict(Hq=260), dict(qs=2552), dict(qs=2564), dict(ks=504), dict(vs=0), dict(ys=2559),
               dict(ks=-512)):
        assert call(**kw) == 2, kw
    for kw in (dict(q=P[0] + 8), dict(k=P[1] + 2), dict(v=P[2] + 4), dict(y=P[5] + 8), dict(cq=P[3] + 2),
               dict(ck=P[4] + 1), dict(lse=P[6] + 2)):
        assert call(**kw) == 3, kw
    # y on top of an input, or inside the span of its strided rows
    assert call(y=P[0]) == 1
    assert call(y=P[1] + 16) == 1
    assert call(v=P[5] + 100 * 2560 * 2 - 16) == 1


def test_decode_refusals(L):
    need = L.bitnet_attn_decode_workspace_size(3, 20, 4, 128)
    assert need > 0
    for bad in ((0, 20, 4, 128), (65537, 20, 4, 128), (3, 20, 3, 128), (3, 20, 4, 32), (3, 65, 1, 128)):
        assert L.bitnet_attn_decode_workspace_size(*bad) == 0

    def call(t=kv(), **kw):
        a = dict(q=P[0], qs=2560, k=P[1], v=P[2], kv=t, slots=None, B=3, Hq=20, Hkv=4, D=128, scale=0.1, y=P[5], ys=2560,
                 lse=None, ws=P[6], nb=need)
        a.update(kw)
        return L.bitnet_attn_decode(*a.values(), None)

    for name in ("q", "k", "v", "kv", "y"):
        assert call(**{name: None}) == 1, name
    for kw, want in BAD_KV:
        assert call(kv(**kw)) == want, kw
    assert call(scale=0.0) == 1
    for kw in (dict(B=0), dict(B=5), dict(Hq=21), dict(D=80), dict(qs=2544), dict(ys=2561)):
        assert call(**kw) == 2, kw
    for kw in (dict(q=P[0] + 2), dict(k=P[1] + 8), dict(slots=P[7] + 2), dict(lse=P[7] + 1), dict(ws=P[6] + 8)):
        assert call(**kw) == 3, kw
    for kw in (dict(y=P[0]), dict(y=P[1] + 64), dict(y=P[2] + 16)):
        assert call(**kw) == 1, kw
    assert call(ws=None) == 4 and call(nb=need - 1) == 4


def test_cache_refusals(L):
    nb = L.bitnet_kv_workspace_size(4, 32)
    assert nb >= 4 * (4 + 2 * 32) and L.bitnet_kv_workspace_size(0, 32) == 0 and L.bitnet_kv_workspace_size(4, 0) == 0
    assert L.bitnet_kv_workspace_size(65537, 32) == 0

    calls = {
        "extend": lambda t=kv(), slots=None, add=P[0], n=3, short=None, ws=P[1], nb=nb: L.bitnet_kv_extend(
            t, slots, add, n, short, ws, nb, None),
        "fork": lambda t=kv(), par=P[0], kid=P[2], n=3, pairs=P[3], np_=P[4], short=None, ws=P[1], nb=nb: L.bitnet_kv_fork(
            t, par, kid, n, pairs, np_, short, ws, nb, None),
        "free": lambda t=kv(), slots=P[0], n=3: L.bitnet_kv_free(t, slots, n, None),
        "compact": lambda t=kv(), pairs=P[3], np_=P[4], live=None, ws=P[1], nb=nb: L.bitnet_kv_compact(
            t, pairs, np_, live, ws, nb, None),
        "append": lambda t=kv(), k=P[0], ks=512, v=P[1], vs=512, cu=P[2], slots=None, B=3, T=9, H=4, D=128, kp=P[3],
        vp=P[4]: L.bitnet_kv_append(k, ks, v, vs, cu, slots, B, T, H, D, t, kp, vp, None),
    }
    for name, call in calls.items():
        assert call(t=None) == 1, name
        for kw, want in BAD_KV:
            assert call(t=kv(**kw)) == want, (name, kw)
    for name, kw, want in [
            ("extend", dict(add=None), 1), ("extend", dict(n=0), 2), ("extend", dict(n=5), 2), ("extend", dict(add=P[0] + 2), 3),
            ("extend", dict(short=P[5] + 1), 3), ("extend", dict(ws=None), 4), ("extend", dict(nb=nb - 1), 4),
            ("extend", dict(ws=P[1] + 4), 3),
            ("fork", dict(par=None), 1), ("fork", dict(kid=None), 1), ("fork", dict(pairs=None), 1), ("fork", dict(np_=None), 1),
            ("fork", dict(n=0), 2), ("fork", dict(n=5), 2), ("fork", dict(kid=P[2] + 2), 3), ("fork", dict(ws=None), 4),
            ("free", dict(slots=None), 1), ("free", dict(n=0), 2), ("free", dict(slots=P[0] + 1), 3),
            ("compact", dict(pairs=None), 1), ("compact", dict(np_=None), 1), ("compact", dict(live=P[5] + 2), 3),
            ("compact", dict(nb=0), 4),
            ("append", dict(k=None), 1), ("append", dict(cu=None), 1), ("append", dict(kp=None), 1), ("append", dict(B=0), 2),
            ("append", dict(B=5), 2), ("append", dict(T=0), 2), ("append", dict(D=72), 2), ("append", dict(ks=508), 2),
            ("append", dict(vs=256), 2), ("append", dict(k=P[0] + 2), 3), ("append", dict(vp=P[4] + 8), 3),
            ("append", dict(kp=P[4]), 1), ("append", dict(k=P[3] + 32), 1), ("append", dict(v=P[4] + 32), 1)]:
        assert calls[name](**kw) == want, (name, kw)

    one = ctypes.c_void_p * 2

    def copy(n=2, k=one(P[0], P[1]), v=one(P[2], P[3]), pages=32, nbytes=4096, pairs=P[4], np_=P[5], most=4):
        return L.bitnet_kv_copy_pages(n, k, v, pages, nbytes, pairs, np_, most, None)

    assert copy(n=0) == 1 and copy(k=None) == 1 and copy(v=one(P[0], None)) == 1 and copy(pairs=None) == 1
    assert copy(np_=None) == 1
    for kw in (dict(pages=0), dict(nbytes=0), dict(nbytes=24), dict(most=0), dict(most=33)):
        assert copy(**kw) == 2, kw
    assert copy(k=one(P[0], P[1] + 8)) == 3 and copy(pairs=P[4] + 2) == 3


def test_binding_refuses_host_tensors_and_wrong_shapes():
    q = torch.zeros(4, 4, 64, dtype=torch.bfloat16)
    c = torch.zeros(2, dtype=torch.int32)
    with pytest.raises(ValueError):
        B.bitnet_attn_prompt(q, q, q, c)
    with pytest.raises(ValueError):
        B.bitnet_kv_pool(4, 4, 8, 16, device="cpu")
    with pytest.raises(ValueError):
        B.bitnet_kv_pool(0, 4, 8, 16, device="cpu")
    with pytest.raises(ValueError):
        B.bitnet_kv_copy_pages([], [], c, c)


def test_scales_whose_product_with_log2_e_is_not_finite(L):
    need = L.bitnet_attn_decode_workspace_size(1, 8, 8, 64)
    for s in (2.5e38, 3.4e38, -2.5e38):
        assert L.bitnet_attn_prompt(P[0], 512, P[1], 512, P[2], 512, P[3], P[4], 1, 9, 9, 8, 8, 64, s, P[5], 512, None, None) == 1
        assert L.bitnet_attn_decode(P[0], 512, P[1], P[2], kv(), None, 1, 8, 8, 64, s, P[5], 512, None, P[6], need, None) == 1


def test_binding_refuses_host_pages_and_pools_of_host_buffers(monkeypatch):
    """Tensors that are all on the host agree with each other about their device; no pointer of theirs may reach the
    library."""
    def called(*a):
        raise AssertionError("the library was called")

    class Fake:
        def __getattr__(self, name):
            return called

    monkeypatch.setattr(B, "_lib", Fake())
    pages = [torch.zeros(6, 2, 16, 64, dtype=torch.bfloat16) for _ in range(2)]
    pairs, n = torch.zeros(3, 2, dtype=torch.int32), torch.zeros(1, dtype=torch.int32)
    with pytest.raises(ValueError):
        B.bitnet_kv_copy_pages(pages[:1], pages[1:], pairs, n)
    with pytest.raises(ValueError):
        B.KvPool(torch.zeros(4 * 8 + 4 + 32, dtype=torch.int32), 4, 8, 32, 16)


def test_binding_imports_without_the_private_names_of_torch():
    """A torch built without CUDA lacks them; the refusals above need none of them."""
    code = ("import torch\n"
            "for n in ('_cuda_getCurrentRawStream', '_cuda_getDevice'):\n"
            "    if hasattr(torch._C, n): delattr(torch._C, n)\n"
            "from ternary_weight_linear_int8_b200 import bitnet as B\n"
            "q = torch.zeros(4, 4, 64, dtype=torch.bfloat16)\n"
            "try: B.bitnet_attn_prompt(q, q, q, torch.zeros(2, dtype=torch.int32))\n"
            "except ValueError: print('refused')\n")
    got = subprocess.run([sys.executable, "-c", code], cwd=os.path.dirname(os.path.dirname(os.path.abspath(__file__))),
                         capture_output=True, text=True, timeout=300)
    assert got.returncode == 0 and got.stdout.strip() == "refused", got.stderr[-2000:]


def test_oracle_row_against_direct_sums():
    rng = np.random.default_rng(0)
    q, k, v = rng.standard_normal(8), rng.standard_normal((5, 8)), rng.standard_normal((5, 8))
    y, lse, ty, tl = A.row(q, k, v, 0.5)
    e = [math.exp(0.5 * sum(a * b for a, b in zip(q, r))) for r in k]
    assert math.isclose(lse, math.log(sum(e)), rel_tol=1e-12)
    want = [sum(w * r[d] for w, r in zip(e, v)) / sum(e) for d in range(8)]
    assert np.allclose(y, want, rtol=1e-12)
    assert (ty > 0).all() and tl > 0
    # no key, and no key with a finite score
    assert A.row(q, k[:0], v[:0], 0.5)[1] == -math.inf
    y, lse, _, _ = A.row(np.abs(q), np.full((3, 8), -math.inf), v[:3], 0.5)
    assert lse == -math.inf and (y == 0).all()
    y = A.row(q, k, np.where(np.arange(5)[:, None] == 2, math.nan, v), 0.5)[0]
    assert np.isnan(y).all()


def test_oracle_prompt_sees_the_causal_border():
    q = np.ones((5, 2, 4))
    k = np.zeros((7, 1, 4))
    v = np.arange(7.0)[:, None, None] * np.ones((1, 1, 4))
    got = {(t, h): y[0] for t, h, y, *_ in A.prompt(q, k, v, [0, 3, 5], [0, 3, 7], 1.0)}
    assert [got[t, 0] for t in range(5)] == [0.0, 0.5, 1.0, 4.0, 4.5]      # second: 2 rows, 4 keys (values 3 .. 6)
    got = [y[0] for _, _, y, *_ in A.prompt(q[:3, :1], k[:1], v[:1], [0, 3], [0, 1], 1.0)]
    assert got == [0.0, 0.0, 0.0]


def test_oracle_pool_takes_lowest_pages_and_shares():
    p = A.Pool(4, 4, 6, 16)
    assert p.extend([20, 5]) == 0
    assert p.table[0].tolist() == [0, 1, -1, -1] and p.table[1].tolist() == [2, -1, -1, -1]
    assert p.extend([60], [2]) == 1 and p.extend([1, 1], [3, 3]) == -1 and p.extend([65], [3]) == -1
    st, pairs = p.fork([0], [3])
    assert st == 0 and pairs == [(1, 3)] and p.table[3].tolist() == [0, 3, -1, -1] and p.refs.tolist() == [2, 1, 1, 1, 0, 0]
    assert p.fork([0], [3])[0] == -1 and p.fork([0, 2], [2, 2])[0] == -1
    p.free([1, 1, 0])
    assert p.refs.tolist() == [1, 0, 0, 1, 0, 0]
    live, pairs = p.compact()
    assert live == 2 and pairs == [(3, 1)] and p.table[3].tolist() == [0, 1, -1, -1]
    assert p.lens.tolist() == [0, 0, 0, 20]
