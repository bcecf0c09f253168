"""Workloads of the attention and key-value cache operators, measured one pass at a time.

Sizes are those of the library's own layers: 2B-class heads (2560-wide query projection: 20 heads of 128; 512-wide
key and value projections: 4 heads), 100B-class heads (8192 wide: 64 heads of 128, 8 key-value heads), and generic
ones with 64-wide heads.  With `own` false a pass computes the operator from elementary torch operations in 32 bits;
with `own` true it makes the library's calls.
"""
import math

import numpy as np
import torch

own = False

BF = torch.bfloat16


def listed():
    return [
        # prompts of a few chat turns batched together: latency counts, a single token and an empty sequence among them
        dict(name="prompt_chat", op="prompt", q_lens="33,1,0,129,64", k_lens="33,1,0,129,64", hq=20, hkv=4, d=128, pad=0),
        # the 4096-token prefill of the 2B-class model, one layer
        dict(name="prompt_prefill_2b", op="prompt", q_lens="4096", k_lens="4096", hq=20, hkv=4, d=128, pad=0),
        # a packed serving batch of uneven prompts at the 100B-class head layout, rows kept beyond the last sequence
        dict(name="prompt_packed_100b", op="prompt", q_lens="2048,77,1,1500,513,3001,400", k_lens="2048,77,1,1500,513,3001,400",
             hq=64, hkv=8, d=128, pad=13),
        # later pieces of long prompts against all keys so far (a piece after a prefix), one key head per query head, 64 wide
        dict(name="prompt_pieces_d64", op="prompt", q_lens="1000,1,700", k_lens="5000,900,700", hq=16, hkv=16, d=64, pad=0),
        # one user's decode step early in a chat
        dict(name="decode_one_short", op="decode", lens="203", hq=20, hkv=4, d=128, page=16, spread=1),
        # a decode step of 16 users of the 2B-class model, uneven contexts
        dict(name="decode_batch_2b", op="decode", lens="4096,1,333,2047,1025,64,3500,17,0,900,2600,128,511,1800,4000,77", hq=20, hkv=4,
             d=128, page=64, spread=1),
        # one user with a very long context: the cache is read by the whole card
        dict(name="decode_one_long", op="decode", lens="100003", hq=64, hkv=8, d=128, page=64, spread=1),
        # a full serving batch at the 100B-class layout
        dict(name="decode_serving_100b", op="decode", lens=",".join(str(1 + (i * 1327) % 4096) for i in range(96)), hq=64, hkv=8,
             d=128, page=32, spread=2),
        # the rows of one decode step of 64 users go into their pages
        dict(name="append_step", op="append", lens=",".join(str(1 + (i * 97) % 1500) for i in range(64)), add=",".join(["1"] * 64), hkv=4,
             d=128, page=16, pages=8192),
        # a packed prefill of uneven prompts goes into fresh pages
        dict(name="append_prefill", op="append", lens="0,0,100,0,2049", add="4096,1,3000,777,8000", hkv=8, d=128, page=64, pages=1024),
        # sampling several continuations of each prompt: the children share full pages, the last one is copied in all layers
        dict(name="fork_samples", op="fork", slots=96, parents=12, children=48, mean=700, hkv=4, d=128, page=64, pages=1200, layers=12),
        # half of the users leave: their pages are freed and the pool is compacted, in all layers
        dict(name="release_compact", op="release", slots=64, leave=32, mean=900, hkv=4, d=128, page=64, pages=1400, layers=12),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    hq, hkv, d = rng.choice([(20, 4, 128), (64, 8, 128), (16, 16, 64), (8, 1, 64), (12, 2, 128), (14, 2, 64), (32, 4, 128)])
    op = rng.choice(["prompt", "prompt", "decode", "decode", "append", "fork", "release"])
    if op == "prompt":
        n = rng.choice([1, 1, 2, 3, 5, 9])
        ql = [_log(rng, 1, 4096 // n) for _ in range(n)]
        kl = [q + rng.choice([0, 0, 0, rng.randint(1, 1500), -rng.randint(0, q - 1)]) for q in ql]   # fewer keys: empty rows
        return dict(op=op, q_lens=",".join(map(str, ql)), k_lens=",".join(map(str, kl)), hq=hq, hkv=hkv, d=d, pad=rng.choice([0, 0, 1, 30]))
    if op == "decode":
        n = rng.choice([1, 2, 4, 7, 16, 33, 64])
        return dict(op=op, lens=",".join(str(_log(rng, 1, min(65536, 200000 // n))) for _ in range(n)), hq=hq, hkv=hkv, d=d,
                    page=rng.choice([16, 32, 48, 64, 128]), spread=rng.choice([1, 2]))
    if op == "append":
        n = rng.choice([1, 3, 8, 32, 100])
        page = rng.choice([16, 32, 48, 64, 128])
        lens = [rng.choice([0, _log(rng, 1, 2000)]) for _ in range(n)]
        add = [1] * n if rng.random() < 0.5 else [_log(rng, 1, 12000 // n) for _ in range(n)]
        pages = sum(-(-(a + b) // page) for a, b in zip(lens, add)) + rng.randint(1, 300)
        return dict(op=op, lens=",".join(map(str, lens)), add=",".join(map(str, add)), hkv=hkv, d=d, page=page, pages=pages)
    page, slots, mean = rng.choice([16, 32, 64, 128]), _log(rng, 8, 96), _log(rng, 40, 900)
    pages = slots * (2 * mean // page + 2)
    layers = max(1, min(rng.randint(1, 12), int(4e8 // (pages * page * hkv * d))))
    if op == "fork":
        parents = max(1, slots // 8)
        return dict(op=op, slots=slots, parents=parents, children=rng.randint(1, slots - parents), mean=mean, hkv=hkv, d=d, page=page,
                    pages=pages, layers=layers)
    return dict(op=op, slots=slots, leave=rng.randint(1, slots - 1), mean=mean, hkv=hkv, d=d, page=page, pages=pages, layers=layers)


def _ints(text):
    return [int(x) for x in text.split(",")]


def _i32(values):
    return torch.tensor(values, dtype=torch.int32, device="cuda")


def _rows(g, n, heads, d, spread=1.0):
    return (torch.randn((n, heads, d), generator=g, device="cuda") * spread).to(BF)


def _cu(lens):
    return np.concatenate([[0], np.cumsum(lens)]).tolist()


def _tables(lens, slots, max_pages, pages, page, rng):
    """Page table, lengths and reference counts of `slots` sequences on shuffled pages of the pool."""
    table = np.full((slots, max_pages), -1, np.int32)
    refs = np.zeros(pages, np.int32)
    order = rng.permutation(pages)
    at = 0
    for b, n in enumerate(lens):
        k = -(-n // page)
        table[b, :k] = order[at:at + k]
        refs[order[at:at + k]] = 1
        at += k
    full = np.zeros(slots, np.int32)
    full[:len(lens)] = lens
    return table, full, refs


class _Pool:
    """The tables as plain tensors (the library's pool has the same members)."""

    def __init__(self, table, lens, refs, page_size):
        self.table, self.lens, self.refs, self.page_size = table, lens, refs, page_size

    def clone(self):
        return _Pool(self.table.clone(), self.lens.clone(), self.refs.clone(), self.page_size)


def _pool(table, lens, refs, page):
    if own:
        from ternary_weight_linear_int8_b200 import bitnet as B
        pool = B.bitnet_kv_pool(table.shape[0], table.shape[1], len(refs), page)
        pool.table.copy_(torch.from_numpy(table))
        pool.lens.copy_(torch.from_numpy(lens))
        pool.refs.copy_(torch.from_numpy(refs))
        return pool
    return _Pool(torch.from_numpy(table).cuda(), torch.from_numpy(lens).cuda(), torch.from_numpy(refs).cuda(), page)


def _caches(g, shape):
    return [torch.empty(shape, dtype=BF, device="cuda").normal_(generator=g) for _ in range(2)]


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    rng = np.random.default_rng(seed)
    op, d, hkv = case["op"], case["d"], case["hkv"]
    s = dict(case)
    if op == "prompt":
        ql, kl = _ints(case["q_lens"]), _ints(case["k_lens"])
        tq, tk, hq = sum(ql) + case["pad"], sum(kl) + case["pad"], case["hq"]
        s.update(ql=ql, kl=kl, q=_rows(g, tq, hq, d, 1.5), k=_rows(g, tk, hkv, d, 1.5), v=_rows(g, tk, hkv, d), cu_q=_i32(_cu(ql)),
                 cu_k=_i32(_cu(kl)), y=torch.zeros((tq, hq, d), dtype=BF, device="cuda"), scale=d ** -0.5)
    elif op == "decode":
        lens, page = _ints(case["lens"]), case["page"]
        need = [-(-n // page) for n in lens]
        pages = sum(need) * case["spread"] + 3
        s.update(pool=_pool(*_tables(lens, len(lens), max(1, max(need)), pages, page, rng), page), scale=d ** -0.5)
        s["k"], s["v"] = _caches(g, (pages, hkv, page, d))
        s["q"] = _rows(g, len(lens), case["hq"], d, 2.0)
        s["y"] = torch.zeros_like(s["q"])
        if own:
            from ternary_weight_linear_int8_b200 import bitnet as B
            s["ws"] = torch.empty(B.bitnet_attn_decode_workspace_size(len(lens), case["hq"], hkv, d), dtype=torch.uint8, device="cuda")
    elif op == "append":
        lens, add, page = _ints(case["lens"]), _ints(case["add"]), case["page"]
        most = max(-(-(a + b) // page) for a, b in zip(lens, add))
        s.update(pool=_pool(*_tables(lens, len(lens), most, case["pages"], page, rng), page), new=_i32(add), cu=_i32(_cu(add)))
        s["k"], s["v"] = _caches(g, (case["pages"], hkv, page, d))
        s["k_new"], s["v_new"] = _rows(g, sum(add), hkv, d), _rows(g, sum(add), hkv, d)
    else:
        page, slots, mean = case["page"], case["slots"], case["mean"]
        held = case["parents"] if op == "fork" else slots
        lens = [int(x) for x in rng.integers(max(1, mean // 2), mean + mean // 2 + 1, held)]
        s["pool"] = _pool(*_tables(lens, slots, 2 * mean // page + 2, case["pages"], page, rng), page)
        s["k"], s["v"] = _caches(g, (case["layers"], case["pages"], hkv, page, d))
        if op == "fork":
            s["parents_of"] = _i32(rng.integers(0, held, case["children"]))
            s["new_slots"] = _i32(held + rng.permutation(slots - held)[:case["children"]])
        else:
            s["leaving"] = _i32(rng.permutation(slots)[:case["leave"]])
        s["k_layers"], s["v_layers"] = list(s["k"].unbind(0)), list(s["v"].unbind(0))
    return s


def _attend(q, k, v, scale, seen):
    """Softmax attention in 32 bits: q [h, m, d], k and v [h, n, d], seen [m, n] or [h, m, n] truth values."""
    x = torch.matmul(q, k.transpose(-1, -2)).mul_(scale)
    x.masked_fill_(~seen, -torch.inf)
    top = x.amax(-1, keepdim=True).clamp_(min=torch.finfo(torch.float32).min)
    p = x.sub_(top).exp_()
    total = p.sum(-1, keepdim=True)
    return torch.matmul(p, v).div_(total.masked_fill(total == 0, 1.0))


def _plain_prompt(s):
    y, g, hkv, d = s["y"], s["hq"] // s["hkv"], s["hkv"], s["d"]
    a = b = 0
    for m, n in zip(s["ql"], s["kl"]):      # one packed sequence at a time: work between sequences would be thrown away
        if m:
            q = s["q"][a:a + m].float().view(m, hkv, g, d).permute(1, 2, 0, 3).reshape(hkv, g * m, d)
            k, v = (s[x][b:b + n].float().transpose(0, 1) for x in ("k", "v"))
            row = torch.arange(m, device="cuda").repeat(g)[:, None]
            o = _attend(q, k, v, s["scale"], torch.arange(n, device="cuda")[None] <= row + (n - m))
            y[a:a + m] = o.view(hkv, g, m, d).permute(2, 0, 1, 3).reshape(m, hkv * g, d).to(BF)
        a, b = a + m, b + n
    return y


def _plain_decode(s):
    p, hkv, g, d = s["pool"], s["hkv"], s["hq"] // s["hkv"], s["d"]
    n = p.table.shape[0]
    at = p.table.clamp(min=0).long()
    k, v = (s[x][at].permute(0, 2, 1, 3, 4).reshape(n * hkv, -1, d).float() for x in ("k", "v"))
    seen = torch.arange(k.shape[1], device="cuda")[None] < p.lens[:, None]
    seen = seen[:, None].expand(n, hkv, -1).reshape(n * hkv, 1, -1)
    o = _attend(s["q"].float().view(n * hkv, g, d), k, v, s["scale"], seen)
    s["y"].copy_(o.view(n, hkv * g, d))
    return s["y"]


def _plain_append(s):
    p, page = s["pool"].clone(), s["page"]
    lens = p.lens + s["new"]
    have = (p.table >= 0).sum(1)
    need = ((lens + page - 1) // page - have).clamp(min=0)
    fresh = torch.nonzero(p.refs == 0)[:int(need.sum()), 0]
    slot = torch.repeat_interleave(torch.arange(len(need), device="cuda"), need)
    nth = torch.arange(len(fresh), device="cuda") - (need.cumsum(0) - need)[slot]
    p.table[slot, have[slot] + nth] = fresh.int()
    p.refs[fresh] = 1
    row = torch.repeat_interleave(torch.arange(len(need), device="cuda"), s["new"].long())
    pos = torch.arange(len(row), device="cuda") - s["cu"][row] + p.lens[row]
    p.lens = lens
    at = p.table[row, pos // page].long()
    s["k"][at, :, pos % page] = s["k_new"]
    s["v"][at, :, pos % page] = s["v_new"]
    return p


def _plain_fork(s):
    p, page = s["pool"].clone(), s["page"]
    par, kid = s["parents_of"].long(), s["new_slots"].long()
    n = p.lens[par]
    rows, full, rest = p.table[par], n // page, n % page > 0
    share = torch.arange(rows.shape[1], device="cuda")[None] < full[:, None]
    p.refs += torch.bincount(rows[share].long(), minlength=len(p.refs)).int()
    fresh = torch.nonzero(p.refs == 0)[:int(rest.sum()), 0]
    kept = torch.where(share, rows, -1)
    kept[rest, full[rest].long()] = fresh.int()
    src = rows[rest, full[rest].long()].long()
    p.table[kid] = kept
    p.lens[kid] = n
    p.refs[fresh] = 1
    s["k"][:, fresh] = s["k"][:, src]
    s["v"][:, fresh] = s["v"][:, src]
    return p


def _plain_release(s):
    p, gone = s["pool"].clone(), s["leaving"].long()
    rows = p.table[gone]
    p.refs -= torch.bincount(rows[rows >= 0].long(), minlength=len(p.refs)).int()
    p.table[gone] = -1
    p.lens[gone] = 0
    live = int((p.refs > 0).sum())
    src = torch.nonzero(p.refs[live:] > 0)[:, 0] + live
    dst = torch.nonzero(p.refs[:live] == 0)[:, 0]
    to = torch.arange(len(p.refs), device="cuda", dtype=torch.int32)
    to[src] = dst.int()
    p.table = torch.where(p.table >= 0, to[p.table.clamp(min=0).long()], p.table)
    p.refs[dst] = p.refs[src]
    p.refs[src] = 0
    s["k"][:, dst] = s["k"][:, src]
    s["v"][:, dst] = s["v"][:, src]
    return p


def _all(s, p):
    return {"table": p.table, "lens": p.lens, "refs": p.refs, "k": s["k"], "v": s["v"]}


def run(s):
    op = s["op"]
    if not own:
        if op == "prompt":
            return _plain_prompt(s)
        if op == "decode":
            return _plain_decode(s)
        return _all(s, {"append": _plain_append, "fork": _plain_fork, "release": _plain_release}[op](s))
    from ternary_weight_linear_int8_b200 import bitnet as B
    if op == "prompt":
        return B.bitnet_attn_prompt(s["q"], s["k"], s["v"], s["cu_q"], s["cu_k"], scale=s["scale"], y=s["y"])[0]
    if op == "decode":
        return B.bitnet_attn_decode(s["q"], s["k"], s["v"], s["pool"], scale=s["scale"], y=s["y"], workspace=s["ws"])[0]
    p = s["pool"].clone()
    if op == "append":
        B.bitnet_kv_extend(p, s["new"])
        B.bitnet_kv_append(s["k_new"], s["v_new"], s["cu"], p, s["k"], s["v"])
    else:
        if op == "fork":
            pairs, n_pairs = B.bitnet_kv_fork(p, s["parents_of"], s["new_slots"])
        else:
            B.bitnet_kv_free(p, s["leaving"])
            pairs, n_pairs = B.bitnet_kv_compact(p)
        B.bitnet_kv_copy_pages(s["k_layers"], s["v_layers"], pairs, n_pairs)
    return _all(s, p)


def _seen_pairs(m, n):
    """Pairs (row, key) with key <= row + n - m, rows 0 .. m-1, keys 0 .. n-1."""
    first = max(0, m - n)                   # rows before it see nothing
    rows = m - first
    return rows * (first + n - m + 1) + rows * (rows - 1) // 2


def work(case):
    d, hkv = case["d"], case["hkv"]
    if case["op"] == "prompt":
        ql, kl = _ints(case["q_lens"]), _ints(case["k_lens"])
        pairs = sum(_seen_pairs(m, n) for m, n in zip(ql, kl))
        return {"bytes": 2 * d * (2 * case["hq"] * sum(ql) + 2 * hkv * sum(kl)), "flops": 4 * d * case["hq"] * pairs}
    if case["op"] == "decode":
        lens = _ints(case["lens"])
        return {"bytes": 2 * d * (2 * case["hq"] * len(lens) + 2 * hkv * sum(lens)) + 4 * sum(-(-n // case["page"]) for n in lens),
                "flops": 4 * d * case["hq"] * sum(lens)}
    row = 2 * d * hkv                       # bytes of one token's keys (or values) in one layer
    if case["op"] == "append":
        lens, add = _ints(case["lens"]), _ints(case["add"])
        return {"bytes": 4 * row * sum(add) + 4 * (case["pages"] + 3 * len(lens)), "flops": 0}
    held = case["mean"] / case["page"] + 0.5   # pages of a sequence, on average
    if case["op"] == "fork":
        moved, entries = case["children"], 2 * case["children"] * held
    else:                                   # pages of those who stay that lie above the new end of the pool
        live = (case["slots"] - case["leave"]) * held
        moved, entries = live * max(0.0, 1 - live / case["pages"]), 2 * case["slots"] * held
    return {"bytes": int(4 * row * case["page"] * case["layers"] * moved + 4 * (entries + 2 * case["pages"])), "flops": 0}


def _exact_rows(q, k, v, scale, shift):
    """One head in 64 bits: row r sees keys 0 .. r + shift.  The weights come from exp(x - log of the sum)."""
    out = torch.zeros((q.shape[0], v.shape[1]), dtype=torch.float64, device="cuda")
    lo = max(0, -shift)
    if lo < q.shape[0] and k.shape[0]:
        x = (q[lo:].double() * scale) @ k.double().T
        x += torch.triu(torch.full_like(x, -torch.inf), diagonal=lo + shift + 1)
        out[lo:] = torch.exp(x - torch.logsumexp(x, dim=1, keepdim=True)) @ v.double()
    return out


def exact(case, seed):
    s = prepare(case, seed)
    op, page = case["op"], case.get("page")
    if op == "prompt":
        y = torch.zeros(s["q"].shape, dtype=torch.float64, device="cuda")
        a = b = 0
        for m, n in zip(s["ql"], s["kl"]):
            for h in range(case["hq"]):
                kh = h // (case["hq"] // case["hkv"])
                y[a:a + m, h] = _exact_rows(s["q"][a:a + m, h], s["k"][b:b + n, kh], s["v"][b:b + n, kh], s["scale"], n - m)
            a, b = a + m, b + n
        return y
    table, lens, refs = (t.cpu().numpy().copy() for t in (s["pool"].table, s["pool"].lens, s["pool"].refs))
    if op == "decode":
        y = torch.zeros(s["q"].shape, dtype=torch.float64, device="cuda")
        g = case["hq"] // case["hkv"]
        for b, n in enumerate(lens.tolist()):
            use = torch.from_numpy(table[b, :-(-n // page)]).long().cuda()
            for kh in range(case["hkv"] if n else 0):
                k, v = (s[x][use, kh].reshape(-1, case["d"])[:n] for x in ("k", "v"))
                x = (s["q"][b, kh * g:(kh + 1) * g].double() * s["scale"]) @ k.double().T
                y[b, kh * g:(kh + 1) * g] = torch.exp(x - torch.logsumexp(x, dim=1, keepdim=True)) @ v.double()
        return y
    k, v = s["k"], s["v"]

    def take():
        return int(np.flatnonzero(refs == 0)[0])

    if op == "append":
        cu = _cu(_ints(case["add"]))
        for b, extra in enumerate(_ints(case["add"])):
            for i in range(-(-int(lens[b]) // page), -(-(int(lens[b]) + extra) // page)):
                table[b, i] = take()
                refs[table[b, i]] = 1
            pos = np.arange(lens[b], lens[b] + extra)
            at = torch.from_numpy(table[b, pos // page].astype(np.int64) * page + pos % page).cuda()
            for h in range(case["hkv"]):
                for cache, new in ((k, s["k_new"]), (v, s["v_new"])):
                    plane = cache[:, h].reshape(-1, case["d"])
                    plane[at] = new[cu[b]:cu[b + 1], h]
                    cache[:, h] = plane.view(-1, page, case["d"])
            lens[b] += extra
    elif op == "fork":
        moves = []
        for a, b in zip(s["parents_of"].tolist(), s["new_slots"].tolist()):
            full = int(lens[a]) // page
            table[b, :full] = table[a, :full]
            np.add.at(refs, table[a, :full], 1)
            lens[b] = lens[a]
            if lens[a] % page:
                table[b, full] = take()
                refs[table[b, full]] = 1
                moves.append((int(table[a, full]), int(table[b, full])))
        for x, y in moves:
            k[:, y], v[:, y] = k[:, x].clone(), v[:, x].clone()
    else:
        for b in s["leaving"].tolist():
            for x in table[b][table[b] >= 0]:
                refs[x] -= 1
            table[b], lens[b] = -1, 0
        live = int((refs > 0).sum())
        for x in range(live, len(refs)):
            if refs[x] > 0:
                y = take()
                k[:, y], v[:, y] = k[:, x].clone(), v[:, x].clone()
                table[table == x] = y
                refs[y], refs[x] = refs[x], 0
    return {"table": torch.from_numpy(table), "lens": torch.from_numpy(lens), "refs": torch.from_numpy(refs), "k": k, "v": v}
