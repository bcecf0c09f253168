"""GPU tests of the attention operators and of the key-value cache against the 64-bit definitions in
oracle/attention.py.  Tolerances are the bounds derived there; integers are equal."""
from __future__ import annotations

import numpy as np
import pytest
import torch

from oracle import attention as A
from ternary_weight_linear_int8_b200 import bitnet as B
from ternary_weight_linear_int8_b200 import inputs
from tests.gpu_util import guarded

pytestmark = pytest.mark.gpu

BF = torch.bfloat16
NAN, INF = float("nan"), float("inf")


@pytest.fixture(autouse=True)
def _status_clean():
    yield
    assert B.bitnet_last_device_status() == 0


def rand(rng, *shape, scale=1.0):
    return torch.from_numpy(rng.standard_normal(shape) * scale).to(BF)


def f64(t):
    return t.double().numpy()


def i32(values):
    return torch.tensor(values, dtype=torch.int32, device="cuda")


def cu(lens, first=0):
    return (first + np.concatenate([[0], np.cumsum(lens)])).tolist()


def check_row(y, lse, want, where):
    wy, wl, ty, tl = want
    bad = np.isnan(wy)
    assert np.array_equal(np.isnan(y), bad), where
    inf = np.isinf(wy)
    assert np.array_equal(y[inf], wy[inf]), where
    fin = np.isfinite(wy)
    off = np.abs(y[fin] - wy[fin]) - ty[fin]
    assert off.size == 0 or off.max() <= 0, (where, off.max(), ty[fin].max())
    if lse is not None and not np.isnan(wl):
        assert lse == wl if np.isinf(wl) else abs(lse - wl) <= tl, (where, lse, wl, tl)


def run_prompt(q, k, v, cq, ck, scale=None, rows=None, lse=True):
    """Runs the kernel on guarded outputs and checks rows (all, or those of `rows`), and that rows outside the
    sequences keep the sentinel."""
    Tq, Hq, D = q.shape
    out, lg = guarded((Tq, Hq, D), BF), guarded((Tq, Hq), torch.float32)
    before = out.t.view(torch.int16).cpu().clone()
    scale = D ** -0.5 if scale is None else scale
    y, l2 = B.bitnet_attn_prompt(q.cuda(), k.cuda(), v.cuda(), i32(cq), i32(ck), scale=scale, y=out.t,
                                 lse=lg.t if lse else None)
    torch.cuda.synchronize()
    out.check()
    lg.check()
    yh, lh = y.double().cpu().numpy(), lg.t.cpu().numpy()
    for token, h, *want in A.prompt(f64(q), f64(k), f64(v), cq, ck, scale, rows):
        check_row(yh[token, h], lh[token, h] if lse else None, want, (token, h))
    inside = np.zeros(Tq, bool)
    for i in range(len(cq) - 1):
        inside[cq[i]:cq[i + 1]] = True
    raw = y.view(torch.int16).cpu()
    assert torch.equal(raw[~inside], before[~inside])
    return y


# (Hq, Hkv, D), query and key lengths
PROMPTS = [
    ((20, 4, 128), [1], [1]),
    ((20, 4, 128), [33, 1, 0, 129, 64], None),
    ((20, 4, 128), [0, 0, 3], None),
    ((4, 4, 64), [63, 64, 65, 127, 128, 129], None),
    ((2, 1, 128), [255, 256, 257], None),
    ((7, 1, 64), [100, 37], None),
    ((12, 4, 128), [200], [391]),
    ((16, 1, 64), [5, 40], [700, 40]),
    ((64, 1, 128), [19], [83]),
    ((33, 1, 64), [30, 2], [30, 130]),
    ((3, 3, 128), [513], None),
    ((8, 2, 128), [70, 10, 5], [20, 0, 1]),          # more rows than keys: rows that see nothing
    ((8, 2, 64), [300, 2], [150, 1]),
    ((10, 2, 128), [1, 1, 1, 1], [1, 128, 129, 4]),  # single tokens after a prefix
]


@pytest.mark.parametrize("heads,ql,kl", PROMPTS)
def test_prompt_matches_definition(heads, ql, kl):
    Hq, Hkv, D = heads
    kl = ql if kl is None else kl
    rng = np.random.default_rng(sum(ql) * 7 + Hq)
    cq, ck = cu(ql), cu(kl)
    q, k, v = rand(rng, cq[-1], Hq, D, scale=2.0), rand(rng, max(1, ck[-1]), Hkv, D, scale=1.5), \
        rand(rng, max(1, ck[-1]), Hkv, D)
    run_prompt(q, k, v, cq, ck)


# long enough on average (over 256 keys a sequence) for the tensor-core kernel: tiles of one and of two halves, borders
# inside and at the ends of steps, groups that do not divide 128, sequences that are empty or see nothing
TILES = [
    ((20, 4, 128), [257], None),
    ((20, 4, 128), [1200, 0, 1, 130], None),
    ((4, 4, 64), [320, 319, 321], None),
    ((2, 1, 128), [255, 256, 257, 640], None),
    ((7, 1, 64), [700], None),
    ((12, 4, 128), [100, 3], [1000, 3]),
    ((16, 1, 64), [5, 40], [700, 40]),
    ((64, 1, 128), [19], [583]),
    ((33, 1, 64), [30, 2], [30, 1130]),
    ((48, 1, 128), [9, 1], [901, 64]),
    ((3, 3, 128), [513], None),
    ((8, 2, 128), [700, 10, 5], [900, 0, 1]),
    ((8, 2, 64), [900, 2], [600, 1]),                # the first 300 rows see nothing
    ((8, 2, 128), [600], [300]),                     # whole tiles see nothing
    ((10, 2, 128), [1, 1, 1, 1], [640, 128, 129, 1024]),
    ((64, 8, 128), [1000, 300], None),
    ((64, 8, 64), [129, 1], [1025, 500]),
]


def some_rows(ql):
    """Rows at the borders of tiles and halves of any group, and a few others."""
    keep = set()
    for n in ql:
        for at in (0, 2, 3, 8, 16, 25, 32, 50, 64, 127, 128, 250, 255, 256, 300, 512, n // 2, n):
            keep |= {at - 1, at, at + 1}
    return keep


@pytest.mark.parametrize("heads,ql,kl", TILES)
def test_prompt_tiles_match_definition(heads, ql, kl):
    Hq, Hkv, D = heads
    kl = ql if kl is None else kl
    assert sum(kl) > 256 * len(kl)
    rng = np.random.default_rng(sum(ql) * 5 + Hq + D)
    cq, ck = cu(ql), cu(kl)
    q, k, v = rand(rng, cq[-1], Hq, D, scale=2.0), rand(rng, ck[-1], Hkv, D, scale=1.5), rand(rng, ck[-1], Hkv, D)
    run_prompt(q, k, v, cq, ck, rows=some_rows(ql))


@pytest.mark.parametrize("D", [64, 128])
def test_prompt_tiles_leave_what_is_outside(D):
    rng = np.random.default_rng(D + 1)
    Hq, Hkv, ql, kl = 10, 2, [310, 0, 9], [900, 0, 9]
    cq, ck = cu(ql, first=5), cu(kl, first=3)
    q, k, v = rand(rng, cq[-1] + 40, Hq, D), rand(rng, ck[-1] + 150, Hkv, D), rand(rng, ck[-1] + 150, Hkv, D)
    for t, c in ((q, cq), (k, ck), (v, ck)):
        t[:c[0]] = NAN
        t[c[-1]:] = INF
    run_prompt(q, k, v, cq, ck, rows=some_rows(ql))


@pytest.mark.parametrize("D,bad", [(64, NAN), (128, NAN), (128, INF), (64, -INF)])
@pytest.mark.parametrize("where", ["v", "k", "q"])
def test_prompt_tiles_poison(D, bad, where):
    rng = np.random.default_rng(31)
    Hq, Hkv, n = 4, 2, 500
    q, k, v = rand(rng, n, Hq, D).abs(), rand(rng, n, Hkv, D), rand(rng, n, Hkv, D)
    dict(q=q, k=k, v=v)[where][397, 1, 5] = bad
    run_prompt(q, k, v, [0, n], [0, n], lse=where == "v", rows={0, 1, 255, 300, 383, 384, 395, 396, 397, 398, 420, 499})


@pytest.mark.parametrize("D", [64, 128])
def test_prompt_tiles_extreme_scores(D):
    rng = np.random.default_rng(32)
    n, low = 520, torch.finfo(BF).min
    rows = {0, 1, 63, 64, 65, 130, 255, 256, 400, 519}
    q, k, v = rand(rng, n, 2, D).abs() + 0.5, rand(rng, n, 1, D), rand(rng, n, 1, D)
    k[3::5] = low
    run_prompt(q, k, v, [0, n], [0, n], lse=False, rows=rows)
    k[:] = low
    y, lse = B.bitnet_attn_prompt(q.cuda(), k.cuda(), v.cuda(), i32([0, n]), want_lse=True)
    assert bool((y == 0).all()) and bool((lse == -INF).all())
    run_prompt(q * 8, rand(rng, n, 1, D, scale=40.0), v, [0, n], [0, n], rows=rows)
    # scores that grow by more than the reference's slack at every step, and ones that only fall
    for sign in (1, -1):
        ramp = (sign * torch.arange(n, dtype=torch.float32)[:, None, None] * 0.05).expand(n, 1, D).to(BF)
        run_prompt(torch.ones(n, 5, D, dtype=BF), ramp, v, [0, n], [0, n], rows=rows)


@pytest.mark.parametrize("heads,ql,kl", [((20, 4, 128), [1500], [1500]), ((16, 16, 64), [700, 300], [2500, 300]),
                                         ((64, 8, 128), [1100, 900], [1100, 900])])
def test_prompt_long_sampled_rows(heads, ql, kl):
    Hq, Hkv, D = heads
    rng = np.random.default_rng(Hq)
    cq, ck = cu(ql), cu(kl)
    rows = {0, 1, 50, 51, 127, 128, 255, 256, 640, -1, -2, -129}
    run_prompt(rand(rng, cq[-1], Hq, D, scale=2.0), rand(rng, ck[-1], Hkv, D), rand(rng, ck[-1], Hkv, D), cq, ck,
               rows=rows)


@pytest.mark.parametrize("D", [64, 128])
def test_prompt_rows_outside_sequences_and_poison(D):
    """Sequences that start late and end early; everything outside them is NaN or infinite and must not be read into
    a row or written."""
    rng = np.random.default_rng(D)
    Hq, Hkv, ql, kl = 10, 2, [70, 0, 9], [90, 0, 9]
    cq, ck = cu(ql, first=5), cu(kl, first=3)
    q, k, v = rand(rng, cq[-1] + 40, Hq, D), rand(rng, ck[-1] + 150, Hkv, D), rand(rng, ck[-1] + 150, Hkv, D)
    for t, c in ((q, cq), (k, ck), (v, ck)):
        t[:c[0]] = NAN
        t[c[-1]:] = INF
    run_prompt(q, k, v, cq, ck)


@pytest.mark.parametrize("D,bad", [(64, NAN), (128, NAN), (128, INF), (64, -INF)])
@pytest.mark.parametrize("where", ["v", "k"])
def test_prompt_poison_behind_the_causal_border(D, bad, where):
    """A value or key that is not finite changes only the rows that see it."""
    rng = np.random.default_rng(3)
    Hq, Hkv, n = 4, 2, 150
    q, k, v = rand(rng, n, Hq, D).abs(), rand(rng, n, Hkv, D), rand(rng, n, Hkv, D)
    (v if where == "v" else k)[97, 1, 5] = bad
    run_prompt(q, k, v, [0, n], [0, n], lse=where == "v")


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("where,bad", [("v", NAN), ("v", -INF), ("k", NAN), ("q", INF)])
@pytest.mark.parametrize("n", [60, 70])
def test_short_prompt_poison(n, D, where, bad):
    rng = np.random.default_rng(34)
    Hq, Hkv = 4, 2
    q, k, v = rand(rng, n, Hq, D).abs(), rand(rng, n, Hkv, D), rand(rng, n, Hkv, D)
    dict(q=q, k=k, v=v)[where][45, 1, 5] = bad
    run_prompt(q, k, v, [0, n], [0, n], lse=where == "v")


@pytest.mark.parametrize("D", [64, 128])
def test_prompt_extreme_scores(D):
    """Keys of the type's lowest value (scores far below the rest, or overflowing to -inf for every key of a row)."""
    rng = np.random.default_rng(4)
    n, low = 140, torch.finfo(BF).min
    q, k, v = rand(rng, n, 2, D).abs() + 0.5, rand(rng, n, 1, D), rand(rng, n, 1, D)
    k[3::5] = low                       # products overflow to -inf: those keys get no weight
    run_prompt(q, k, v, [0, n], [0, n], lse=False)
    k[:] = low                          # every score -inf: rows give 0
    y = B.bitnet_attn_prompt(q.cuda(), k.cuda(), v.cuda(), i32([0, n]))[0]
    assert bool((y == 0).all())
    k = rand(rng, n, 1, D, scale=40.0)  # sharp: one key holds almost all of the weight
    run_prompt(q * 8, k, v, [0, n], [0, n])


@pytest.mark.parametrize("scale", [1e-40, 1e-20, 3.0, 1e30])
@pytest.mark.parametrize("n", [40, 400])
def test_prompt_scales_from_tiny_to_huge(scale, n):
    """With a vanishing scale every key weighs the same; with a huge one the largest score takes all (its score is 0, so
    that products stay finite)."""
    rng = np.random.default_rng(35)
    q, k, v = rand(rng, n, 4, 64).abs(), -rand(rng, n, 1, 64).abs() - 0.1, rand(rng, n, 1, 64)
    k[::7] = 0
    if scale > 100:
        k[1:] = torch.where(k[1:] == 0, torch.tensor(-1.0, dtype=BF), k[1:])
    y, lse = B.bitnet_attn_prompt(q.cuda(), k.cuda(), v.cuda(), i32([0, n]), scale=scale, want_lse=True)
    yh, lh = y.double().cpu().numpy(), lse.cpu().numpy()
    if scale > 100:                                    # weights 1 for the first key, 0 for the others
        assert np.array_equal(yh, np.broadcast_to(f64(v[0, 0]), yh.shape)) and np.allclose(lh, 0, atol=1e-6)
    else:
        for t, h, *want in A.prompt(f64(q), f64(k), f64(v), [0, n], [0, n], np.float64(np.float32(scale)),
                                    rows={0, 1, 31, 32, 100, 255, 256, n - 1}):
            check_row(yh[t, h], lh[t, h], want, (t, h))


def test_prompt_growing_scores():
    """Scores that grow along the keys move the running maximum at every step."""
    rng = np.random.default_rng(5)
    n, D = 400, 128
    q = torch.ones(n, 5, D, dtype=BF)
    k = (torch.arange(n, dtype=torch.float32)[:, None, None] * 0.03).expand(n, 1, D).to(BF)
    run_prompt(q, k, rand(rng, n, 1, D), [0, n], [0, n])


def test_prompt_fused_projection_strides_and_scale():
    rng = np.random.default_rng(6)
    n, Hq, Hkv, D = 77, 20, 4, 128
    w = (Hq + 2 * Hkv) * D
    buf = rand(rng, n, w + 8).cuda()
    q = buf[:, :Hq * D].view(n, Hq, D)
    k = buf[:, Hq * D:(Hq + Hkv) * D].view(n, Hkv, D)
    v = buf[:, (Hq + Hkv) * D:w].view(n, Hkv, D)
    ybuf = torch.full((n, Hq * D + 16), 7.0, dtype=BF, device="cuda")
    y = ybuf[:, 8:8 + Hq * D].view(n, Hq, D)
    B.bitnet_attn_prompt(q, k, v, i32([0, n]), scale=0.3, y=y)
    yh = y.double().cpu().numpy()
    for t, h, *want in A.prompt(f64(q.cpu()), f64(k.cpu()), f64(v.cpu()), [0, n], [0, n], np.float32(0.3)):
        check_row(yh[t, h], None, want, (t, h))
    assert bool((ybuf[:, :8] == 7).all()) and bool((ybuf[:, 8 + Hq * D:] == 7).all())
    one = B.bitnet_attn_prompt(q[:1], k[:1], v[:1], i32([0, 1]))[0]          # one token: its own value
    assert torch.equal(one[0], v[0].repeat_interleave(Hq // Hkv, 0))


def test_prompt_overlapping_bounds_stay_inside():
    """Bounds that go back and forth: every second sequence is refused, the others overlap; nothing is written outside."""
    rng = np.random.default_rng(36)
    T = 300
    q, k, v = (rand(rng, T, h, 64).cuda() for h in (4, 1, 1))
    out = guarded((T, 4, 64), BF)
    want = B.bitnet_attn_prompt(q, k, v, i32([0, T]))[0]
    B.bitnet_attn_prompt(q, k, v, i32([0, T] * 200), y=out.t)
    assert B.bitnet_last_device_status() == 1
    out.check()
    assert torch.allclose(out.t, want, atol=0.02)


def test_prompt_bad_bounds_are_recorded():
    rng = np.random.default_rng(7)
    q, k, v = (rand(rng, 64, h, 64).cuda() for h in (4, 2, 2))
    out = guarded((64, 4, 64), BF)
    good = B.bitnet_attn_prompt(q, k, v, i32([0, 20, 64]))[0]
    for bad in ([-5, 20, 64], [0, 20, 65], [0, 70, 64], [0, 20, 10]):
        B.bitnet_attn_prompt(q, k, v, i32(bad), y=out.t)
        assert B.bitnet_last_device_status() == 1
        out.check()
    B.bitnet_attn_prompt(q, k, v, i32([0, 20, 64]), i32([0, 20, 65]), y=out.t)
    assert B.bitnet_last_device_status() == 1
    out.check()
    assert torch.equal(out.t[:20], good[:20])           # the sound sequence is computed


def test_prompt_captured_and_replayed_on_new_bounds():
    """A captured call reads the bounds at replay."""
    rng = np.random.default_rng(33)
    T, Hq, Hkv, D = 900, 10, 2, 128
    q, k, v = rand(rng, T, Hq, D), rand(rng, T, Hkv, D), rand(rng, T, Hkv, D)
    qd, kd, vd, c = q.cuda(), k.cuda(), v.cuda(), i32([0, 400, 900])
    y = torch.zeros_like(qd)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        B.bitnet_attn_prompt(qd, kd, vd, c, y=y)
    side.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        B.bitnet_attn_prompt(qd, kd, vd, c, y=y)
    for bounds in ([0, 700, 899], [3, 3, 500]):
        c.copy_(i32(bounds))
        y.fill_(9.0)
        graph.replay()
        yh = y.double().cpu().numpy()
        for t, h, *want in A.prompt(f64(q), f64(k), f64(v), bounds, bounds, D ** -0.5, rows={0, 60, 399, -1, -2}):
            check_row(yh[t, h], None, want, (t, h))
        assert bool((y[:bounds[0]] == 9).all()) and bool((y[bounds[-1]:] == 9).all())


def test_prompt_same_bits_again_on_another_stream():
    rng = np.random.default_rng(8)
    q, k, v = (rand(rng, 900, h, 128).cuda() for h in (20, 4, 4))
    c = i32([0, 300, 900])
    first = B.bitnet_attn_prompt(q, k, v, c)[0]
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        again = B.bitnet_attn_prompt(q, k, v, c)[0]
    s.synchronize()
    assert torch.equal(first.view(torch.int16), again.view(torch.int16))


# ------------------------------------------------------------------ cache
def make_cache(rng, lens, page, Hkv, D, spare=3, poison=NAN, extra_slots=0, max_pages=None):
    """A pool whose sequences lie on shuffled pages; what no sequence holds is `poison`.  Returns (pool, host pool,
    k_pages, v_pages, keys and values of each sequence)."""
    need = [-(-n // page) for n in lens]
    n_pages = sum(need) + spare
    mp = max(1, max(need)) if max_pages is None else max_pages
    host = A.Pool(len(lens) + extra_slots, mp, n_pages, page)
    order = rng.permutation(n_pages)
    kp = torch.full((n_pages, Hkv, page, D), poison, dtype=BF)
    vp = torch.full((n_pages, Hkv, page, D), poison, dtype=BF)
    ks, vs, at = [], [], 0
    for b, n in enumerate(lens):
        pages = order[at:at + need[b]]
        at += need[b]
        host.table[b, :need[b]] = pages
        host.refs[pages] = 1
        host.lens[b] = n
        k, v = rand(rng, n, Hkv, D), rand(rng, n, Hkv, D)
        for i, p in enumerate(pages):
            rows = min(page, n - i * page)
            kp[p, :, :rows] = k[i * page:i * page + rows].transpose(0, 1)
            vp[p, :, :rows] = v[i * page:i * page + rows].transpose(0, 1)
        ks.append(k)
        vs.append(v)
    return to_device(host), host, kp.cuda(), vp.cuda(), ks, vs


def to_device(host):
    pool = B.bitnet_kv_pool(host.table.shape[0], host.table.shape[1], len(host.refs), host.page_size)
    pool.table.copy_(torch.from_numpy(host.table))
    pool.lens.copy_(torch.from_numpy(host.lens))
    pool.refs.copy_(torch.from_numpy(host.refs))
    return pool


def same_tables(pool, host):
    assert np.array_equal(pool.table.cpu().numpy(), host.table)
    assert np.array_equal(pool.lens.cpu().numpy(), host.lens)
    assert np.array_equal(pool.refs.cpu().numpy(), host.refs)


DECODES = [
    ((20, 4, 128), 16, [1]),
    ((20, 4, 128), 16, [0, 1, 15, 16, 17, 63, 64, 65]),
    ((64, 8, 128), 64, [130, 0, 0, 700]),
    ((4, 4, 64), 48, [47, 48, 49, 200, 1]),
    ((8, 1, 64), 1024, [1023, 1025]),
    ((16, 2, 128), 32, [900]),
    ((9, 1, 128), 16, [77, 300]),
    ((16, 1, 64), 16, [1000, 3]),
    ((33, 1, 128), 16, [40, 90]),          # several blocks of query heads
    ((64, 1, 64), 80, [333]),
    ((7, 7, 128), 16, [5, 129]),
    ((40, 2, 64), 16, [0, 0, 0]),
]


@pytest.mark.parametrize("heads,page,lens", DECODES)
def test_decode_matches_definition(heads, page, lens):
    Hq, Hkv, D = heads
    rng = np.random.default_rng(sum(lens) + Hq)
    pool, _, kp, vp, ks, vs = make_cache(rng, lens, page, Hkv, D)
    n = len(lens)
    q = rand(rng, n, Hq, D, scale=2.0)
    out, lg = guarded((n, Hq, D), BF), guarded((n, Hq), torch.float32)
    ws = guarded((B.bitnet_attn_decode_workspace_size(n, Hq, Hkv, D),), torch.uint8)
    y, _ = B.bitnet_attn_decode(q.cuda(), kp, vp, pool, y=out.t, lse=lg.t, workspace=ws.t)
    torch.cuda.synchronize()
    for g in (out, lg, ws):
        g.check()
    yh, lh = y.double().cpu().numpy(), lg.t.cpu().numpy()
    for b in range(n):
        for h in range(Hq):
            want = A.row(f64(q[b, h]), f64(ks[b][:, h // (Hq // Hkv)]), f64(vs[b][:, h // (Hq // Hkv)]), D ** -0.5)
            check_row(yh[b, h], lh[b, h], want, (b, h))


@pytest.mark.parametrize("lens", [[20000], [3, 9000, 1, 0, 4000, 64] * 4])
def test_decode_split_over_the_card(lens):
    """Lengths that several blocks share: sampled heads, and the same bits again."""
    rng = np.random.default_rng(len(lens))
    Hq, Hkv, D = 20, 4, 128
    pool, _, kp, vp, ks, vs = make_cache(rng, lens, 64, Hkv, D)
    q = rand(rng, len(lens), Hq, D, scale=2.0)
    y, lse = B.bitnet_attn_decode(q.cuda(), kp, vp, pool, want_lse=True)
    again = B.bitnet_attn_decode(q.cuda(), kp, vp, pool)[0]
    assert torch.equal(y.view(torch.int16), again.view(torch.int16))
    yh, lh = y.double().cpu().numpy(), lse.cpu().numpy()
    for b in range(len(lens)):
        for h in (0, 4, 5, 13, 19):
            want = A.row(f64(q[b, h]), f64(ks[b][:, h // 5]), f64(vs[b][:, h // 5]), D ** -0.5)
            check_row(yh[b, h], lh[b, h], want, (b, h))


def test_decode_slots_strides_and_shared_slots():
    rng = np.random.default_rng(11)
    Hq, Hkv, D, lens = 8, 2, 64, [30, 100, 1, 0]
    pool, _, kp, vp, ks, vs = make_cache(rng, lens, 32, Hkv, D)
    slots = [1, 1, 3, 0, 2, 1]
    buf = rand(rng, 6, Hq * D + 64).cuda()
    q = buf[:, 32:32 + Hq * D].view(6, Hq, D)
    y = B.bitnet_attn_decode(q, kp, vp, pool, slots=i32(slots), scale=0.2)[0].double().cpu().numpy()
    for b, s in enumerate(slots):
        for h in range(Hq):
            check_row(y[b, h], None, A.row(f64(q[b, h].cpu()), f64(ks[s][:, h // 4]), f64(vs[s][:, h // 4]),
                                           np.float32(0.2)), (b, h))


def test_decode_bad_tables_are_recorded():
    rng = np.random.default_rng(12)
    Hq, Hkv, D, lens = 8, 2, 128, [100, 40]
    pool, host, kp, vp, ks, vs = make_cache(rng, lens, 16, Hkv, D)
    q = rand(rng, 2, Hq, D)
    good = B.bitnet_attn_decode(q.cuda(), kp, vp, pool)[0]
    for page in (-1, 10 ** 6, -7):
        pool.table[0, 3] = page                   # tokens 48 .. 63 are not seen
        y = B.bitnet_attn_decode(q.cuda(), kp, vp, pool)[0]
        assert B.bitnet_last_device_status() == 9
        assert torch.equal(y[1], good[1])
        keep = np.r_[0:48, 64:100]
        for h in range(Hq):
            check_row(y[0, h].double().cpu().numpy(), None,
                      A.row(f64(q[0, h]), f64(ks[0][keep, h // 4]), f64(vs[0][keep, h // 4]), D ** -0.5), h)
    pool.table.copy_(torch.from_numpy(host.table))
    for bad in (-1, 10 ** 6):
        pool.lens[0] = bad
        y = B.bitnet_attn_decode(q.cuda(), kp, vp, pool)[0]
        assert B.bitnet_last_device_status() == 9
        assert bool((y[0] == 0).all()) and torch.equal(y[1], good[1])
    pool.lens[0] = 100
    y = B.bitnet_attn_decode(q.cuda(), kp, vp, pool, slots=i32([-3, 1]))[0]
    assert B.bitnet_last_device_status() == 9
    assert bool((y[0] == 0).all()) and torch.equal(y[1], good[1])


def test_decode_sees_what_is_not_finite():
    """NaN and infinities in seen keys and values act as in the definition."""
    rng = np.random.default_rng(13)
    Hq, Hkv, D, lens = 4, 1, 64, [70]
    for where, bad in (("v", NAN), ("v", INF), ("k", -INF), ("k", NAN)):
        pool, host, kp, vp, ks, vs = make_cache(rng, lens, 16, Hkv, D)
        (ks if where == "k" else vs)[0][20, 0, 9] = bad
        (kp if where == "k" else vp)[int(host.table[0, 1]), 0, 4, 9] = bad
        q = rand(rng, 1, Hq, D).abs()
        y = B.bitnet_attn_decode(q.cuda(), kp, vp, pool)[0].double().cpu().numpy()
        for h in range(Hq):
            check_row(y[0, h], None, A.row(f64(q[0, h]), f64(ks[0][:, 0]), f64(vs[0][:, 0]), D ** -0.5), (where, bad))


def test_cache_offsets_past_32_bits():
    """Pages whose byte and element offsets pass 2^32 and 2^31: append, decode and page copies there."""
    Hkv, page, D = 8, 64, 128
    n_pages = 36000                                # 4.7 GB of keys
    rng = np.random.default_rng(14)
    kp = torch.zeros((n_pages, Hkv, page, D), dtype=BF, device="cuda")
    vp = torch.zeros_like(kp)
    pool = B.bitnet_kv_pool(2, 4, n_pages, page)
    pool.refs.fill_(1)
    pool.refs[-4:] = 0
    B.bitnet_kv_extend(pool, i32([130]))
    k, v, q = rand(rng, 130, Hkv, D), rand(rng, 130, Hkv, D), rand(rng, 2, 16, D)
    B.bitnet_kv_append(k.cuda(), v.cuda(), i32([0, 130]), pool, kp, vp)
    assert pool.table[0].tolist() == [n_pages - 4, n_pages - 3, n_pages - 2, -1]
    pairs, n = B.bitnet_kv_fork(pool, i32([0]), i32([1]))
    B.bitnet_kv_copy_pages([kp], [vp], pairs, n)
    y = B.bitnet_attn_decode(q.cuda(), kp, vp, pool)[0].double().cpu().numpy()
    for b in range(2):
        for h in range(16):
            check_row(y[b, h], None, A.row(f64(q[b, h]), f64(k[:, h // 2]), f64(v[:, h // 2]), D ** -0.5), (b, h))


def test_append_writes_only_its_rows():
    rng = np.random.default_rng(15)
    Hkv, D, page = 3, 64, 16
    for lens, add, first in (([5, 0, 40, 15, 16], [1, 33, 0, 1, 1], 0), ([0], [1], 0), ([31, 7], [2, 50], 4)):
        pool, host, kp, vp, ks, vs = make_cache(rng, lens, page, Hkv, D, spare=12, poison=2.0, max_pages=8)
        T = sum(add) + first + 3
        k, v = rand(rng, T, Hkv, D), rand(rng, T, Hkv, D)
        k[:first], k[first + sum(add):] = NAN, NAN
        B.bitnet_kv_extend(pool, i32(add))
        assert host.extend(add) == 0
        same_tables(pool, host)
        wk, wv = kp.cpu(), vp.cpu()
        c = cu(add, first=first)
        for b, a in enumerate(add):
            for i in range(a):
                pos = host.lens[b] - a + i
                p, r = host.table[b, pos // page], pos % page
                wk[p, :, r], wv[p, :, r] = k[c[b] + i], v[c[b] + i]
        B.bitnet_kv_append(k.cuda(), v.cuda(), i32(c), pool, kp, vp)
        assert torch.equal(kp.cpu(), wk) and torch.equal(vp.cpu(), wv)


def test_append_skips_what_has_no_place():
    rng = np.random.default_rng(16)
    pool, host, kp, vp, _, _ = make_cache(rng, [20, 20], 16, 2, 64, poison=0.0)
    before = kp.clone()
    k = rand(rng, 30, 2, 64).cuda()
    for slots, c in (([0, 7], [0, 0, 1]), ([-1, 1], [0, 1, 1]), ([0, 1], [0, 25, 25])):
        B.bitnet_kv_append(k, k, i32(c), pool, kp, vp, slots=i32(slots))
        assert B.bitnet_last_device_status() == 9
    assert torch.equal(kp[host.table[1, :2].tolist()].cpu(), before[host.table[1, :2].tolist()].cpu())


def random_ops(seed, n_slots, max_pages, n_pages, page, steps, layers=2, Hkv=2, D=64):
    rng = np.random.default_rng(seed)
    host = A.Pool(n_slots, max_pages, n_pages, page)
    pool = to_device(host)
    kp = [torch.from_numpy(rng.standard_normal((n_pages, Hkv, page, D))).to(BF) for _ in range(layers)]
    kd, vd = [t.cuda() for t in kp], [(-t).cuda() for t in kp]
    short, live = i32([99]), i32([99])

    def copies(pairs, n, want):
        assert int(n) == len(want)
        assert pairs[:len(want)].tolist() == [list(p) for p in want]
        B.bitnet_kv_copy_pages(kd, vd, pairs, n)
        for t in kp:
            for a, b in want:
                t[b] = t[a]

    seen = {"refused": 0, "short": 0, "ok": 0}
    for _ in range(steps):
        op = rng.choice(["extend", "extend", "fork", "fork", "free", "compact"])
        if op == "extend":
            slots = rng.choice(n_slots + 1, size=rng.integers(1, n_slots), replace=bool(rng.random() < 0.1)).tolist()
            slots = [s for s in slots if s < n_slots or rng.random() < 0.1] or [0]
            add = rng.integers(0, 3 * page, len(slots)).tolist()
            want = host.extend(add, slots)
            B.bitnet_kv_extend(pool, i32(add), slots=i32(slots), short_pages=short)
        elif op == "fork":
            empty = [s for s in range(n_slots) if host.lens[s] == 0]
            kids = rng.permutation(empty)[:rng.integers(1, 5)].tolist() if empty and rng.random() < 0.9 else [0]
            held = [s for s in range(n_slots) if host.lens[s]] or [1]
            par = rng.choice(held, size=len(kids)).tolist()
            want, pairs = host.fork(par, kids)
            got, n = B.bitnet_kv_fork(pool, i32(par), i32(kids), short_pages=short)
            copies(got, n, pairs)
        elif op == "free":
            slots = rng.integers(0, n_slots, rng.integers(1, 6)).tolist()
            host.free(slots)
            B.bitnet_kv_free(pool, i32(slots))
            want = None
        else:
            used, pairs = host.compact()
            got, n = B.bitnet_kv_compact(pool, live=live)
            assert int(live) == used
            copies(got, n, pairs)
            want = None
        if want is not None:
            assert int(short) == want
            assert B.bitnet_last_device_status() == (0 if want == 0 else 9)
            seen["ok" if want == 0 else "refused" if want < 0 else "short"] += 1
        same_tables(pool, host)
    for t, a, b in zip(kp, kd, vd):
        assert torch.equal(a.cpu(), t) and torch.equal(b.cpu(), -t)
    return seen


@pytest.mark.parametrize("seed,shape", [(1, (12, 8, 60, 16)), (2, (40, 5, 4200, 48)), (3, (3, 20, 9, 16)),
                                        (4, (100, 3, 131, 32))])
def test_page_operations_follow_the_definition(seed, shape):
    seen = random_ops(seed, *shape, steps=60)
    assert seen["ok"]
    if seed in (1, 3):
        assert seen["short"] or seen["refused"]


def test_pool_refusals_change_nothing():
    rng = np.random.default_rng(17)
    pool, host, _, _, _, _ = make_cache(rng, [20, 33, 0, 0], 16, 1, 64, spare=2, max_pages=5)
    short = i32([5])
    for add, slots, want in (([1, 1], [0, 0], -1), ([-1], [0], -1), ([70], [0], -1), ([1], [4], -1), ([1], [-1], -1),
                             ([13, 16, 1], [0, 1, 2], 1), ([80], [3], 3)):
        B.bitnet_kv_extend(pool, i32(add), slots=i32(slots), short_pages=short)
        assert int(short) == want and B.bitnet_last_device_status() == 9
        same_tables(pool, host)
    for par, kid in (([0], [1]), ([0, 0], [2, 2]), ([0], [0]), ([9], [2]), ([0], [-1]), ([0, 2], [2, 3])):
        _, n = B.bitnet_kv_fork(pool, i32(par), i32(kid), short_pages=short)
        assert int(short) == -1 and int(n) == 0 and B.bitnet_last_device_status() == 9
        same_tables(pool, host)
    B.bitnet_kv_free(pool, i32([-1, 9]))
    assert B.bitnet_last_device_status() == 9
    same_tables(pool, host)


def test_binding_refuses_other_types():
    x = torch.zeros(4, 2, 64, device="cuda")
    c = i32([0, 4])
    h = x.to(BF)
    for bad in (x.half(), x, x.to(torch.int32)):
        for args in ((bad, h, h), (h, bad, h), (h, h, bad)):
            with pytest.raises(ValueError):
                B.bitnet_attn_prompt(*args, c)
        with pytest.raises(ValueError):
            B.bitnet_attn_prompt(h, h, h, c, y=bad)
    with pytest.raises(ValueError):
        B.bitnet_attn_prompt(h, h, h, c.long())
    with pytest.raises(ValueError):
        B.bitnet_attn_prompt(h.transpose(1, 2), h, h, c)
    with pytest.raises(B.BitnetError):                 # 96-wide heads
        B.bitnet_attn_prompt(*[torch.zeros(4, 2, 96, dtype=BF, device="cuda")] * 3, c)
    with pytest.raises(B.BitnetError):                 # one row for every token
        B.bitnet_attn_prompt(h[:1].expand(4, 2, 64), h, h, c)
    pool = B.bitnet_kv_pool(2, 2, 4, 16)
    pages = torch.zeros(4, 2, 16, 64, dtype=BF, device="cuda")
    for bad in (pages.half(), pages[:3], pages[:, :, :8], torch.zeros(4, 2, 16, 128, dtype=BF, device="cuda")):
        with pytest.raises(ValueError):
            B.bitnet_attn_decode(h[:2], bad, bad, pool)
        with pytest.raises(ValueError):
            B.bitnet_kv_append(h, h, c, pool, bad, bad)
    with pytest.raises(ValueError):
        B.bitnet_kv_extend(pool, torch.ones(2, device="cuda"))


def test_copy_pages_skips_pairs_outside_the_pool():
    k = torch.arange(8 * 16 * 64, device="cuda").view(8, 1, 16, 64).to(BF)
    v = -k
    want = k.clone()
    want[6] = want[1]
    B.bitnet_kv_copy_pages([k], [v], i32([0, 8, -1, 2, 1, 6, 99, 3]).view(4, 2), i32([9]))   # count beyond the list
    assert B.bitnet_last_device_status() == 9
    assert torch.equal(k, want) and torch.equal(v, -want)
    B.bitnet_kv_copy_pages([k], [v], i32([0, 7]).view(1, 2), i32([0]))
    B.bitnet_kv_copy_pages([k], [v], i32([0, 7]).view(1, 2), i32([-4]))
    assert torch.equal(k, want)


def test_copy_pages_in_many_layers_and_odd_pages():
    rng = np.random.default_rng(18)
    for layers, shape in ((130, (6, 1, 16, 64)), (3, (5, 7, 48, 128))):
        ks = [rand(rng, *shape) for _ in range(layers)]
        kd, vd = [t.cuda() for t in ks], [(t * 2).cuda() for t in ks]
        B.bitnet_kv_copy_pages(kd, vd, i32([0, 3, 1, 4]).view(2, 2), i32([2]))
        for t, a, b in zip(ks, kd, vd):
            t[3], t[4] = t[0], t[1]
            assert torch.equal(a.cpu(), t) and torch.equal(b.cpu(), t * 2)


# ------------------------------------------------------- used together
def test_decode_step_captured_and_replayed():
    """extend, append and decode recorded once: every replay goes by the tables of that moment.  A second graph uses
    the same workspace."""
    rng = np.random.default_rng(19)
    Hq, Hkv, D, lens, page, steps = 10, 2, 128, [15, 0, 100], 16, 20
    pool, host, kp, vp, ks, vs = make_cache(rng, lens, page, Hkv, D, spare=8, max_pages=9)
    one, c = i32([1, 1, 1]), i32([0, 1, 2, 3])
    q, kn, vn = (torch.zeros(3, h, D, dtype=BF, device="cuda") for h in (Hq, Hkv, Hkv))
    ws = torch.empty(B.bitnet_attn_decode_workspace_size(3, Hq, Hkv, D), dtype=torch.uint8, device="cuda")
    y, y2 = torch.empty_like(q), torch.empty_like(q)

    def step():
        B.bitnet_kv_extend(pool, one)
        B.bitnet_kv_append(kn, vn, c, pool, kp, vp)
        B.bitnet_attn_decode(q, kp, vp, pool, y=y, workspace=ws)

    side = torch.cuda.Stream()
    keep = pool.buf.clone()
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        step()                                    # loads the kernels
        pool.buf.copy_(keep)
    side.synchronize()
    graph, other = torch.cuda.CUDAGraph(), torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        step()
    with torch.cuda.graph(other, stream=side):
        B.bitnet_attn_decode(q, kp, vp, pool, y=y2, scale=0.5, workspace=ws)
    for t in range(steps):
        nq, nk, nv = rand(rng, 3, Hq, D), rand(rng, 3, Hkv, D), rand(rng, 3, Hkv, D)
        q.copy_(nq)
        kn.copy_(nk)
        vn.copy_(nv)
        graph.replay()
        other.replay()
        assert host.extend([1, 1, 1]) == 0
        for b in range(3):
            ks[b], vs[b] = torch.cat([ks[b], nk[b:b + 1]]), torch.cat([vs[b], nv[b:b + 1]])
        for yy, scale in ((y, D ** -0.5), (y2, 0.5)):
            yh = yy.double().cpu().numpy()
            for b in range(3):
                for h in range(0, Hq, 3):
                    check_row(yh[b, h], None, A.row(f64(nq[b, h]), f64(ks[b][:, h // 5]), f64(vs[b][:, h // 5]), scale),
                              (t, b, h))
    same_tables(pool, host)


def test_layer_from_projections_to_output():
    """A decoder layer's attention as it is used: q/k/v projections, a packed prompt, its rows into pages, forked
    continuations decoded a few tokens on, some of them freed, the pool compacted, and the output projection.  The
    decoded rows equal prompt attention over the whole sequence within the bounds of both."""
    rng = np.random.default_rng(20)
    H, Hq, Hkv, D, page = 512, 8, 2, 64, 16
    Ws = [inputs.weights(n, H, rng=rng) for n in (Hq * D, Hkv * D, Hkv * D)]
    packs = [B.bitnet_pack_weights(torch.from_numpy(w).cuda()) for w in Ws]
    po, go = B.bitnet_pack_weights(torch.from_numpy(inputs.weights(H, Hq * D, rng=rng)).cuda())

    def qkv(x):
        q, k, v = B.bitnet_linear_multi([p for p, _ in packs], [g for _, g in packs], x)
        n = x.shape[0]
        return q.view(n, Hq, D), k.view(n, Hkv, D), v.view(n, Hkv, D)

    lens = [37, 5, 64]
    pool = B.bitnet_kv_pool(8, 8, 40, page)
    kp, vp = (torch.zeros(40, Hkv, page, D, dtype=BF, device="cuda") for _ in range(2))
    x = rand(rng, sum(lens), H).cuda()
    q, k, v = qkv(x)
    c = i32(cu(lens))
    y = B.bitnet_attn_prompt(q, k, v, c)[0]
    out = B.bitnet_linear(po, go, y.view(-1, Hq * D))[0]
    assert out.shape == (sum(lens), H) and bool(torch.isfinite(out).all())
    B.bitnet_kv_extend(pool, i32(lens), slots=i32([0, 1, 2]))
    B.bitnet_kv_append(k, v, c, pool, kp, vp, slots=i32([0, 1, 2]))
    pairs, n = B.bitnet_kv_fork(pool, i32([0, 2, 0]), i32([3, 4, 5]))
    B.bitnet_kv_copy_pages([kp], [vp], pairs, n)
    at = cu(lens)
    hist = {s: (list(k[at[p]:at[p + 1]].cpu()), list(v[at[p]:at[p + 1]].cpu()))
            for s, p in ((0, 0), (1, 1), (2, 2), (3, 0), (4, 2), (5, 0))}
    active = [0, 1, 2, 3, 4, 5]
    for t in range(20):
        if t == 9:
            B.bitnet_kv_free(pool, i32([0, 4]))
            pairs, n = B.bitnet_kv_compact(pool)
            B.bitnet_kv_copy_pages([kp], [vp], pairs, n)
            active = [5, 1, 3, 2]
        m = len(active)
        slots = i32(active)
        xq, xk, xv = qkv(rand(rng, m, H).cuda())
        B.bitnet_kv_extend(pool, i32([1] * m), slots=slots)
        B.bitnet_kv_append(xk, xv, i32(list(range(m + 1))), pool, kp, vp, slots=slots)
        y = B.bitnet_attn_decode(xq, kp, vp, pool, slots=slots)[0]
        out = B.bitnet_linear(po, go, y.view(m, Hq * D))[0]
        assert bool(torch.isfinite(out).all())
        yh = y.double().cpu().numpy()
        for i, s in enumerate(active):
            hist[s][0].append(xk[i].cpu())
            hist[s][1].append(xv[i].cpu())
            kk, vv = f64(torch.stack(hist[s][0])), f64(torch.stack(hist[s][1]))
            for h in (0, 3, 7):
                check_row(yh[i, h], None, A.row(f64(xq[i, h].cpu()), kk[:, h // 4], vv[:, h // 4], D ** -0.5), (t, s, h))
    refs = pool.refs.cpu().numpy()
    tab = pool.table.cpu().numpy()
    assert np.array_equal(refs, np.bincount(tab[tab >= 0], minlength=40))


def test_two_calls_at_once_on_two_streams():
    """Calls on different streams with their own workspaces do not disturb each other."""
    rng = np.random.default_rng(21)
    Hq, Hkv, D = 20, 4, 128
    pool, _, kp, vp, _, _ = make_cache(rng, [3000, 500, 7], 64, Hkv, D)
    qs = [rand(rng, 3, Hq, D).cuda() for _ in range(2)]
    want = [B.bitnet_attn_decode(q, kp, vp, pool)[0] for q in qs]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    got = [[], []]
    for _ in range(10):
        for i in range(2):
            with torch.cuda.stream(streams[i]):
                got[i].append(B.bitnet_attn_decode(qs[i], kp, vp, pool)[0])
    torch.cuda.synchronize()
    for i in range(2):
        for y in got[i]:
            assert torch.equal(y.view(torch.int16), want[i].view(torch.int16))
