"""GPU tests of the attention and cache operators at the ends of their documented ranges: demands above the pool, damaged
tables and bounds, scores and values at the ends of fp32's range.  Definitions and bounds as in test_gpu_attention.py."""
from __future__ import annotations

import numpy as np
import pytest
import torch

from oracle import attention as A
from ternary_weight_linear_int8_b200 import bitnet as B
from tests import test_gpu_attention as T

pytestmark = pytest.mark.gpu

BF = torch.bfloat16
NAN, INF = float("nan"), float("inf")


@pytest.fixture(autouse=True)
def _status_clean():
    yield
    assert B.bitnet_last_device_status() == 0


# ------------------------------------------------------------------ cache
@pytest.mark.parametrize("add,slots", [([150 * 16], [0]), ([101 * 16], [1]), ([60 * 16, 60 * 16], [0, 1]),
                                       ([1, 200 * 16 - 1, 0], [2, 0, 1])])
def test_extend_wants_more_than_an_empty_pool_has(add, slots):
    host = A.Pool(3, 200, 100, 16)
    pool, short = T.to_device(host), T.i32([77])
    want = host.extend(add, slots)
    assert want > 0
    B.bitnet_kv_extend(pool, T.i32(add), slots=T.i32(slots), short_pages=short)
    assert B.bitnet_last_device_status() == 9
    assert int(short) == want
    T.same_tables(pool, host)
    # exactly all of it is granted afterwards
    assert host.extend([100 * 16], [slots[0]]) == 0
    B.bitnet_kv_extend(pool, T.i32([100 * 16]), slots=T.i32(slots[:1]), short_pages=short)
    assert int(short) == 0
    T.same_tables(pool, host)


def test_extend_more_rows_than_threads():
    host = A.Pool(2300, 3, 4000, 16)
    rng = np.random.default_rng(41)
    pool, short = T.to_device(host), T.i32([77])
    for add in (rng.integers(0, 40, 2300), np.full(2300, 30), np.full(2300, 8)):
        add = np.minimum(add, 48 - host.lens).tolist()
        want = host.extend(add)
        B.bitnet_kv_extend(pool, T.i32(add), short_pages=short)
        assert int(short) == want and B.bitnet_last_device_status() == (9 if want else 0)
        T.same_tables(pool, host)


def test_extend_by_more_pages_than_two_million():
    """One slot that takes 2.5 million pages of a pool of three; the tables alone, no pages behind them."""
    n_pages, entries = 3_000_000, 2_500_000
    pool, short = B.bitnet_kv_pool(2, entries, n_pages, 16), T.i32([77])
    pool.refs[100_000:] = 1                                    # too few are free
    B.bitnet_kv_extend(pool, T.i32([entries * 16]), short_pages=short)
    assert B.bitnet_last_device_status() == 9 and int(short) == entries - 100_000
    assert bool((pool.table == -1).all()) and bool((pool.lens == 0).all()) and int(pool.refs.sum()) == 2_900_000
    pool.refs[100_000:] = 0
    pool.refs[5:10] = 3
    B.bitnet_kv_extend(pool, T.i32([entries * 16 - 3]), short_pages=short)
    assert int(short) == 0 and pool.lens.tolist() == [entries * 16 - 3, 0]
    pages = torch.cat([torch.arange(5), torch.arange(10, entries + 5)]).to(torch.int32)
    assert torch.equal(pool.table[0].cpu(), pages) and bool((pool.table[1] == -1).all())
    refs = torch.zeros(n_pages, dtype=torch.int32)
    refs[:entries + 5] = 1
    refs[5:10] = 3
    assert torch.equal(pool.refs.cpu(), refs)
    # both rows at once want more than 2^21 pages that are not there
    B.bitnet_kv_extend(pool, T.i32([3, entries * 16]), short_pages=short)
    assert B.bitnet_last_device_status() == 9 and int(short) == entries - (n_pages - entries - 5)
    assert pool.lens.tolist() == [entries * 16 - 3, 0] and torch.equal(pool.refs.cpu(), refs)


@pytest.mark.parametrize("c", [[-2_000_000_000, 2_000_000_000], [-2 ** 31, 2 ** 31 - 1], [-2 ** 31, 25, 25],
                               [0, 2 ** 31 - 1], [-1_500_000_000, 700_000_000, 2 ** 31 - 1]])
def test_append_bounds_from_end_to_end_of_int32(c):
    """Bounds whose difference does not fit 32 bits: no row has a position, or only those that the length holds."""
    rng = np.random.default_rng(42)
    pool, host, kp, vp, _, _ = T.make_cache(rng, [20, 20], 16, 2, 64, poison=0.0)
    want = [kp.cpu().clone(), vp.cpu().clone()]
    k = T.rand(rng, 30, 2, 64)
    skipped = False
    for r in range(30):
        b = max(i for i in range(len(c)) if c[i] <= r)
        if b == len(c) - 1:
            continue
        pos = 20 - c[b + 1] + r
        skipped |= pos < 0
        if pos >= 0:
            for w in want:
                w[host.table[b, pos // 16], :, pos % 16] = k[r]
    B.bitnet_kv_append(k.cuda(), k.cuda(), T.i32(c), pool, kp, vp)
    assert B.bitnet_last_device_status() == (9 if skipped else 0)
    assert torch.equal(kp.cpu(), want[0]) and torch.equal(vp.cpu(), want[1])
    T.same_tables(pool, host)


@pytest.mark.parametrize("max_pages", [8, 3000])                # planned and written by one launch, and by two
@pytest.mark.parametrize("bad", [-1, -2 ** 31, "n_pages", 2 ** 31 - 1])
@pytest.mark.parametrize("entry", [0, 1, 3])
def test_fork_of_a_parent_on_a_page_outside_the_pool(max_pages, bad, entry):
    """Entry 3 is the partly filled one.  Nothing changes, in the tables of the sound parent's child neither."""
    rng = np.random.default_rng(43)
    pool, host, _, _, _, _ = T.make_cache(rng, [50, 20, 0, 0], 16, 1, 64, spare=6, max_pages=max_pages)
    host.table[0, entry] = len(host.refs) if bad == "n_pages" else bad
    pool.table.copy_(torch.from_numpy(host.table))
    short = T.i32([77])
    assert host.fork([1, 0], [2, 3]) == (-1, [])
    _, n = B.bitnet_kv_fork(pool, T.i32([1, 0]), T.i32([2, 3]), short_pages=short)
    assert B.bitnet_last_device_status() == 9
    assert int(short) == -1 and int(n) == 0
    T.same_tables(pool, host)
    want, pairs = host.fork([1], [2])
    got, n = B.bitnet_kv_fork(pool, T.i32([1]), T.i32([2]), short_pages=short)
    assert want == 0 and int(short) == 0 and got[:int(n)].tolist() == [list(p) for p in pairs]
    T.same_tables(pool, host)


def test_fork_of_long_parents():
    """Parents of more entries than a warp reads at a time; a bad one at the end of the last of 40 is found."""
    rng = np.random.default_rng(44)
    lens = [int(x) for x in rng.integers(1000, 3000, 40)] + [0] * 50
    pool, host, _, _, _, _ = T.make_cache(rng, lens, 16, 1, 64, spare=60, max_pages=200)
    keep, short = host.table[39].copy(), T.i32([77])
    par, kids = list(range(40)) + [3, 3, 39], list(range(40, 83))
    host.table[39, (lens[39] - 1) // 16] = -1
    pool.table.copy_(torch.from_numpy(host.table))
    B.bitnet_kv_fork(pool, T.i32(par), T.i32(kids), short_pages=short)
    assert B.bitnet_last_device_status() == 9 and int(short) == -1
    T.same_tables(pool, host)
    host.table[39] = keep
    pool.table.copy_(torch.from_numpy(host.table))
    want, pairs = host.fork(par, kids)
    got, n = B.bitnet_kv_fork(pool, T.i32(par), T.i32(kids), short_pages=short)
    assert want == 0 and int(short) == 0 and got[:int(n)].tolist() == [list(p) for p in pairs]
    T.same_tables(pool, host)


def test_append_after_a_refused_extend_is_skipped_by_slots_of_minus_one():
    """A captured step whose slots become -1 on the device where the extend was refused: nothing that is held changes."""
    rng = np.random.default_rng(46)
    pool, host, kp, vp, _, _ = T.make_cache(rng, [31, 16], 16, 2, 64, spare=1, poison=2.0, max_pages=4)
    ids, one, c, short = T.i32([0, 1]), T.i32([1, 1]), T.i32([0, 1, 2]), T.i32([0])
    k = T.rand(rng, 2, 2, 64).cuda()

    def step():
        B.bitnet_kv_extend(pool, one, short_pages=short)
        B.bitnet_kv_append(k, -k, c, pool, kp, vp, slots=torch.where(short == 0, ids, -1).to(torch.int32))

    side = torch.cuda.Stream()
    keep = pool.buf.clone(), kp.clone(), vp.clone()
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        step()
        for t, u in zip((pool.buf, kp, vp), keep):
            t.copy_(u)
    side.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        step()
    for granted in (True, False):                                # slot 1 takes the last page, then slot 0 wants one
        graph.replay()
        assert (host.extend([1, 1]) == 0) == granted
        assert B.bitnet_last_device_status() == (0 if granted else 9) and (int(short) == 0) == granted
        T.same_tables(pool, host)
        if granted:
            held = kp.clone(), vp.clone()
            for b, n in ((0, 32), (1, 17)):
                assert torch.equal(kp[int(host.table[b, (n - 1) // 16]), :, (n - 1) % 16], k[b])
            k.copy_(T.rand(rng, 2, 2, 64))
    assert torch.equal(kp, held[0]) and torch.equal(vp, held[1])


def test_free_of_entries_that_no_count_holds():
    """Damaged tables: pages that are named more often than counted.  Their counts end at 0 and they can be taken again."""
    rng = np.random.default_rng(45)
    pool, host, _, _, _, _ = T.make_cache(rng, [40, 20, 16], 16, 1, 64, spare=3, max_pages=4)
    pool.refs[int(host.table[0, 1])] = 0
    pool.table[1, 0] = int(host.table[0, 2])                     # named twice, counted once
    pool.refs[int(host.table[1, 0])] = 0
    B.bitnet_kv_free(pool, T.i32([0, 1]))
    assert B.bitnet_last_device_status() == 9
    left = torch.zeros(len(host.refs), dtype=torch.int32)
    left[int(host.table[2, 0])] = 1
    assert torch.equal(pool.refs.cpu(), left)
    short = T.i32([77])
    B.bitnet_kv_extend(pool, T.i32([64, 64]), slots=T.i32([0, 1]), short_pages=short)
    assert int(short) == 0 and bool((pool.refs == 1).all())


# ------------------------------------------------------------- scores
def check_far(y, lse, q, keys, vals, scale, where):
    """A row whose q . k are exact in fp32 (small integers).  What the kernels round then is the exponent: scale * log2 e,
    the difference of two scores where they are not close, and its product, half a step each, and 2^-22 of the exponential;
    a key whose exponent is below -40 has no weight that shows.  Sums of n terms add n U_SUM, a weight half a bf16 step.
    The log-sum adds two rounded products of the scale."""
    n = len(keys)
    s = keys @ q * scale
    top = s.max()
    p = np.exp(s - top)
    total = p.sum()
    rel = 40 * 3 * 2.0 ** -24 + 2.0 ** -22 + (n + 8) * A.U_SUM
    want = (p[:, None] * vals).sum(0) / total
    spread = (p[:, None] * np.abs(vals)).sum(0) / total
    assert np.all(np.abs(y - want) <= spread * (A.U_BF16 + 2 * rel) * 1.01 + np.abs(want) * A.U_BF16), where
    if abs(top) < 3.402e38:                                          # fp32 ends at 3.4028e38
        assert abs(lse - (top + np.log(total))) <= abs(top) * 2.0 ** -22 + rel + 2.0 ** -20, (where, lse, top)
    elif abs(top) > 3.404e38:
        assert lse == np.sign(top) * np.inf, (where, lse, top)


SCALES = [2.0 ** 20, 2.0 ** 26, 1.5e9, 2.0 ** 34, 1e12, 1e20, 1e30, 2e36, 2.3e38]


@pytest.mark.parametrize("scale", SCALES)
@pytest.mark.parametrize("sign", [1, -1])
@pytest.mark.parametrize("n,D", [(40, 64), (40, 128), (400, 64), (400, 128)])       # both sides of the dispatch rule
def test_prompt_scores_far_from_zero(n, D, sign, scale):
    """The largest score is far from 0, above or below: the row is the mean of the values of the keys that share it."""
    rng = np.random.default_rng(50)
    scale = float(np.float32(scale))
    q = torch.from_numpy(rng.integers(1, 4, (n, 4, D))).to(BF)
    k = torch.from_numpy(sign * rng.integers(0, 4, (n, 2, D))).to(BF)
    k[:, 0] = k[torch.from_numpy(rng.integers(0, 6, n)), 0]          # ties
    k[0, 0, 0] = k[0, 1, 0] = sign * 3.0
    v = T.rand(rng, n, 2, D)
    y, lse = B.bitnet_attn_prompt(q.cuda(), k.cuda(), v.cuda(), T.i32([0, n]), scale=scale, want_lse=True)
    yh, lh = y.double().cpu().numpy(), lse.double().cpu().numpy()
    qh, kh, vh = T.f64(q), T.f64(k), T.f64(v)
    for t in range(0, n, 1 if n < 100 else 7):
        for h in range(4):
            check_far(yh[t, h], lh[t, h], qh[t, h], kh[:t + 1, h // 2], vh[:t + 1, h // 2], scale, (t, h))


@pytest.mark.parametrize("scale", SCALES[:-2])                     # scale * q . k stays in fp32's range
@pytest.mark.parametrize("sign", [1, -1])
@pytest.mark.parametrize("lens,heads", [([5, 70, 1, 400], (4, 2, 64)), ([20000, 3], (20, 2, 128))])
def test_decode_scores_far_from_zero(lens, heads, sign, scale):
    rng = np.random.default_rng(51)
    Hq, Hkv, D = heads
    scale = float(np.float32(scale))
    pool, host, kp, vp, ks, vs = T.make_cache(rng, lens, 64, Hkv, D)
    for b, n in enumerate(lens):
        ks[b] = torch.from_numpy(sign * rng.integers(0, 4, (n, Hkv, D))).to(BF)
        ks[b][:, 0] = ks[b][torch.from_numpy(rng.integers(0, min(n, 6), n)), 0]
        ks[b][0, :, 0] = sign * 3.0
        for i in range(-(-n // 64)):
            rows = min(64, n - i * 64)
            kp[int(host.table[b, i]), :, :rows] = ks[b][i * 64:i * 64 + rows].transpose(0, 1).cuda()
    q = torch.from_numpy(rng.integers(1, 4, (len(lens), Hq, D))).to(BF)
    y, lse = B.bitnet_attn_decode(q.cuda(), kp, vp, pool, scale=scale, want_lse=True)
    yh, lh = y.double().cpu().numpy(), lse.double().cpu().numpy()
    for b in range(len(lens)):
        kh, vh = T.f64(ks[b]), T.f64(vs[b])
        for h in range(0, Hq, 3):
            g = h // (Hq // Hkv)
            check_far(yh[b, h], lh[b, h], T.f64(q[b, h]), kh[:, g], vh[:, g], scale, (b, h))


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("bad", [NAN, INF, -INF])
def test_prompt_scores_far_from_zero_and_keys_that_are_not_finite(D, bad):
    """Rows that see the key and rows that do not, scores that come from far below 0 to near it, and back up."""
    rng = np.random.default_rng(52)
    n = 400
    q = torch.ones(n, 2, D, dtype=BF)
    k = torch.zeros(n, 1, D, dtype=BF)
    k[:, 0, 0] = torch.tensor([-2.0 ** 34] * 70 + [-2.0 ** 33] * 70 + [-3.0] * 70 + [1.0] * 70 + [2.0 ** 35] * 50 + [0.0] * 70)
    k[360, 0, 1] = bad
    v = T.rand(rng, n, 1, D)
    y, lse = B.bitnet_attn_prompt(q.cuda(), k.cuda(), v.cuda(), T.i32([0, n]), scale=1.0, want_lse=True)
    yh, lh = y.double().cpu().numpy(), lse.double().cpu().numpy()
    kh, vh = T.f64(k), T.f64(v)
    kh[360, 0, 1] = -np.inf if bad == -INF else 0.0      # no weight for the rows that are checked, or not seen by them
    for t in list(range(0, n if bad == -INF else 360, 3)):
        for h in range(2):
            seen = [j for j in range(t + 1) if j != 360]
            check_far(yh[t, h], lh[t, h], np.ones(D), kh[seen, 0], vh[seen, 0], 1.0, (t, h))
    if bad != -INF:
        assert np.isnan(yh[360:]).all()


# ------------------------------------------------ values that are not finite
def poisoned(rng, n, Hkv, D, places):
    """Values with the given (position, head, column or None for all, value) written over them."""
    v = T.rand(rng, n, Hkv, D)
    for at, h, d, x in places:
        v[at, h, slice(None) if d is None else d] = x
    return v


# by column: what a row sees first, what lies behind its border, one or both infinities, all of a column, all of a row
POISON = [
    [(3, 0, 5, NAN), (200, 0, 7, NAN), (201, 0, 5, INF)],
    [(3, 0, None, NAN)],
    [(3, 0, 5, INF), (3, 0, 9, -INF), (230, 0, 5, -INF), (231, 0, 9, NAN)],
    [(slice(None), 0, 11, INF), (slice(None), 1, None, NAN)],
    [(slice(None), 1, 2, -INF), (100, 1, 2, NAN), (250, 0, None, INF), (251, 0, None, -INF)],
    [(slice(40, None, 3), 0, 60, NAN), (slice(41, None, 3), 1, 1, INF)],
]


@pytest.mark.parametrize("places", POISON)
@pytest.mark.parametrize("n,D", [(60, 64), (60, 128), (300, 64), (300, 128), (520, 128)])
def test_prompt_values_that_are_not_finite(n, D, places):
    rng = np.random.default_rng(60)
    keep = [p for p in places if isinstance(p[0], slice) or p[0] < n]
    v = poisoned(rng, n, 2, D, keep)
    q, k = T.rand(rng, n, 4, D), T.rand(rng, n, 2, D)
    rows = {0, 1, 2, 3, 4, 39, 40, 41, 42, 59, 99, 100, 101, 127, 128, 129, 185, 199, 200, 201, 202, 229, 230, 231, 232, 249,
            250, 251, 252, 299, 400, 519}
    T.run_prompt(q, k, v, [0, n], [0, n], rows=rows)


@pytest.mark.parametrize("n,D", [(50, 64), (50, 128), (400, 64), (400, 128)])
def test_prompt_values_at_the_end_of_the_range(n, D):
    """Equal values of 2^127 and of half of it: their weighted sum before the division is past fp32's range."""
    rng = np.random.default_rng(61)
    q, k = T.rand(rng, n, 4, D, scale=0.1), T.rand(rng, n, 2, D)
    v = T.rand(rng, n, 2, D)
    v[:, 0, 3], v[:, 1, 0], v[5:, 1, 7] = 2.0 ** 127, -2.0 ** 126, 2.0 ** 127
    T.run_prompt(q, k, v, [0, n], [0, n], rows={0, 1, 2, 10, 49, 127, 128, 399})


@pytest.mark.parametrize("n,D", [(50, 64), (50, 128), (400, 64), (400, 128)])
@pytest.mark.parametrize("bad", [NAN, INF])
def test_prompt_rows_without_weight_are_zero_whatever_the_values(n, D, bad):
    rng = np.random.default_rng(62)
    q, k, v = T.rand(rng, n, 4, D).abs() + 0.5, T.rand(rng, n, 2, D), T.rand(rng, n, 2, D)
    k[:, 0] = -INF
    k[:30, 1] = -INF
    v[7], v[n - 2, :, 3] = bad, bad
    T.run_prompt(q, k, v, [0, n], [0, n])


@pytest.mark.parametrize("lens", [[70, 3], [9000, 64]])            # one block a head, and joined ones
@pytest.mark.parametrize("bad", [NAN, INF])
def test_decode_rows_without_weight_are_zero_whatever_the_values(lens, bad):
    rng = np.random.default_rng(63)
    Hq, Hkv, D = 8, 2, 64
    pool, host, kp, vp, ks, vs = T.make_cache(rng, lens, 16, Hkv, D)
    kp[:, 0] = -INF
    ks = [k.clone() for k in ks]
    for k in ks:
        k[:, 0] = -INF
    for b, n in enumerate(lens):
        at = n // 2
        vs[b][at] = bad
        vp[int(host.table[b, at // 16]), :, at % 16] = bad
    q = T.rand(rng, 2, Hq, D).abs() + 0.5
    y, lse = B.bitnet_attn_decode(q.cuda(), kp, vp, pool, want_lse=True)
    yh, lh = y.double().cpu().numpy(), lse.cpu().numpy()
    for b in range(2):
        for h in range(Hq):
            T.check_row(yh[b, h], lh[b, h], A.row(T.f64(q[b, h]), T.f64(ks[b][:, h // 4]), T.f64(vs[b][:, h // 4]), D ** -0.5),
                        (b, h))


# ------------------------------------------------------ dispatch of prompts
@pytest.mark.parametrize("heads,ql,kl", [
    ((20, 4, 128), [5, 0, 31, 64, 1, 27], None), ((20, 4, 128), [5, 0, 31, 64, 1, 28], None),     # 128 keys in all, and more
    ((8, 1, 64), [63, 64, 65, 0, 64], None), ((8, 1, 64), [63, 64, 65, 1, 64], None),             # 256
    ((12, 2, 128), [3, 9, 1], [64, 9, 40]), ((16, 16, 64), [30, 7], [100, 100]),
    ((8, 1, 64), [0] * 19 + [1000], None), ((8, 1, 64), [0] * 5 + [200] + [0] * 14, None),        # one sequence has it all
    ((12, 2, 128), [0] * 10 + [128] + [0] * 9, None), ((20, 4, 128), [0] * 3 + [300], None)])
def test_prompt_short_and_uneven_batches(heads, ql, kl):
    Hq, Hkv, D = heads
    kl = ql if kl is None else kl
    rng = np.random.default_rng(sum(ql) + D)
    cq, ck = T.cu(ql), T.cu(kl)
    T.run_prompt(T.rand(rng, cq[-1], Hq, D, scale=2.0), T.rand(rng, ck[-1], Hkv, D), T.rand(rng, ck[-1], Hkv, D), cq, ck,
                 rows=None if max(ql) < 200 else T.some_rows(ql))


@pytest.mark.parametrize("heads,n", [((8, 1, 64), 1200), ((12, 2, 128), 700)])
def test_prompt_one_long_sequence_among_empty_ones_is_no_slower(heads, n):
    """Where it lies among empty sequences does not send a long prompt to the kernel for very short ones.  Shortest
    device times of the two calls in turn; the kernel for short prompts takes 1.6 times as long, a search over 20 bounds a few percent."""
    Hq, Hkv, D = heads
    q, k, v = (torch.randn(n, h, D, device="cuda").to(BF) for h in (Hq, Hkv, Hkv))
    y = torch.empty_like(q)
    cs = [T.i32([0, n]), T.i32([0] * 8 + [n] * 13)]
    graphs = []
    for c in cs:
        B.bitnet_attn_prompt(q, k, v, c, y=y)
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            for _ in range(20):
                B.bitnet_attn_prompt(q, k, v, c, y=y)
        graphs.append(g)
    times = [[], []]
    for _ in range(15):
        for g, t in zip(graphs, times):
            a, b = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
            a.record()
            g.replay()
            b.record()
            b.synchronize()
            t.append(a.elapsed_time(b))
    one, many = (min(t) for t in times)
    assert many < 1.35 * one, (one, many)


def test_binding_without_the_private_names_of_torch(monkeypatch):
    """The public calls that stand in for them give the same stream and device."""
    rng = np.random.default_rng(64)
    q, k, v = (T.rand(rng, 90, h, 64).cuda() for h in (4, 2, 2))
    c = T.i32([0, 40, 90])
    want = B.bitnet_attn_prompt(q, k, v, c)[0]
    monkeypatch.setattr(B, "_raw_stream", lambda dev: torch.cuda.current_stream(dev).cuda_stream)
    monkeypatch.setattr(B, "_current_device", torch.cuda.current_device)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        got = B.bitnet_attn_prompt(q, k, v, c)[0]
    side.synchronize()
    assert torch.equal(got.view(torch.int16), want.view(torch.int16))
