"""The serving operators around the decode step, as cases to measure: rows of whole prompts written into the
caches, causal attention over packed prompts, attention of a batch that shares prefixes, forking of sequences on
shared pages, and compaction of a page pool.

`own` chooses between the plain form (elementary torch operations) and the library's calls.
"""
import math
import random

import numpy as np
import torch

own = False

DEV = "cuda"


def listed():
    return [
        # sixteen requests in flight, each with a piece of its prompt, behind what is cached already
        dict(name="append_ragged", op="append", B=16, Hq=32, Hkv=8, d=128, bs=64, paged=True, new_lo=1, new_hi=512,
             old_lo=0, old_hi=4096, mix=3),
        # the whole 32K prompt of one request
        dict(name="append_32k", op="append", B=1, Hq=32, Hkv=8, d=128, bs=128, paged=False, new_lo=32768,
             new_hi=32768, old_lo=0, old_hi=0, mix=0),
        # one short question: latency counts
        dict(name="prompt_tiny", op="prompt", B=1, Hq=4, Hkv=1, d=64, bs=64, paged=True, new_lo=37, new_hi=37,
             old_lo=0, old_hi=0, mix=0),
        # an ordinary mixed batch, single tokens and prompts of some thousand packed together
        dict(name="prompt_ragged", op="prompt", B=16, Hq=32, Hkv=8, d=128, bs=64, paged=True, new_lo=1, new_hi=4096,
             old_lo=0, old_hi=0, mix=1),
        # pieces of two long prompts behind a long cached context
        dict(name="prompt_chunk", op="prompt", B=2, Hq=64, Hkv=8, d=128, bs=128, paged=True, new_lo=1000, new_hi=1024,
             old_lo=60000, old_hi=65536, mix=2),
        # a whole 32K prompt
        dict(name="prompt_32k", op="prompt", B=1, Hq=32, Hkv=8, d=128, bs=64, paged=False, new_lo=32768, new_hi=32768,
             old_lo=0, old_hi=0, mix=0),
        # eight short conversations on two common instructions
        dict(name="shared_8x4k", op="shared", B=8, Hq=4, Hkv=1, d=64, bs=64, paged=True, groups=2, prefix=4096,
             own_lo=1, own_hi=64, mix=4),
        # sixty-four samples of four long documents
        dict(name="shared_64x128k", op="shared", B=64, Hq=64, Hkv=8, d=128, bs=128, paged=True, groups=4,
             prefix=131072, own_lo=1, own_hi=2048, mix=5),
        # four samples of one short prompt are dropped and drawn anew
        dict(name="fork_1x4", op="fork", parents=1, children=4, Hq=4, Hkv=1, d=64, bs=64, ctx_lo=4000, ctx_hi=4090,
             spare=8, mix=6),
        # fifteen samples of each of four long documents
        dict(name="fork_4x15", op="fork", parents=4, children=15, Hq=32, Hkv=8, d=128, bs=128, ctx_lo=100000,
             ctx_hi=131072, spare=64, mix=7),
        # a small pool after some requests ended
        dict(name="compact_256", op="compact", B=8, pages=256, live=150, Hq=4, Hkv=1, d=64, bs=64, mix=8),
        # a large pool, half of it free
        dict(name="compact_8192", op="compact", B=16, pages=8192, live=4096, Hq=32, Hkv=8, d=128, bs=128, mix=9),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["append", "prompt", "prompt", "shared", "shared", "fork", "compact"])
    Hkv = rng.choice([1, 2, 4, 8])
    G = rng.choice([1, 2, 3, 4, 5, 7, 8])
    c = dict(op=op, Hq=Hkv * G, Hkv=Hkv, d=rng.choice([64, 128]), bs=rng.choice([64, 128]), mix=rng.randrange(1 << 30))
    if op == "append":
        B = _log(rng, 1, 32)
        hi = _log(rng, 1, 32768 // B)
        c.update(B=B, paged=rng.random() < 0.6, new_lo=rng.choice([1, _up(hi, 2), hi]), new_hi=hi, old_lo=0,
                 old_hi=_log(rng, 1, 4096))
    elif op == "prompt":
        B = _log(rng, 1, 24)
        hi = _log(rng, 1, (16384 if Hkv * G <= 32 else 8192) // B)
        c.update(B=B, paged=rng.random() < 0.6, new_lo=rng.choice([1, _up(hi, 2), hi]), new_hi=hi, old_lo=0,
                 old_hi=_log(rng, 1, 16384 if B < 4 else 4096))
    elif op == "shared":
        groups = rng.randint(1, 4)
        c.update(B=groups * _log(rng, 1, 16), paged=rng.random() < 0.7, groups=groups,
                 prefix=c["bs"] * _log(rng, 1, 32768 // c["bs"]), own_lo=1, own_hi=_log(rng, 1, 2048))
    elif op == "fork":
        hi = _log(rng, 128, 65536)
        c.update(parents=rng.randint(1, 4), children=_log(rng, 1, 15), ctx_lo=max(1, hi // 2), ctx_hi=hi,
                 spare=rng.randint(1, 64))
    else:
        pages = _log(rng, 16, 4096)
        c.update(B=rng.randint(1, 16), pages=pages, live=rng.randint(1, pages))
    return c


# ----------------------------------------------------------------------------- what a case is made of

def _lengths(c):
    """(new, old) rows of each sequence, by the case alone."""
    r = random.Random(c["mix"])
    new = [_log(r, c["new_lo"], c["new_hi"]) for _ in range(c["B"])]
    old = [r.randint(c["old_lo"], c["old_hi"]) for _ in range(c["B"])]
    return new, old


def _own_lengths(c):
    r = random.Random(c["mix"])
    return [_log(r, c["own_lo"], c["own_hi"]) for _ in range(c["B"])]


def _contexts(c):
    r = random.Random(c["mix"])
    return [r.randint(c["ctx_lo"], c["ctx_hi"]) for _ in range(c["parents"])]


def _up(a, b):
    return -(-a // b)


def _gen(seed):
    return torch.Generator(device=DEV).manual_seed(seed)


def _randn(g, *shape):
    return torch.randn(shape, generator=g, device=DEV, dtype=torch.bfloat16)


def _i32(x):
    return torch.tensor(np.asarray(x), dtype=torch.int32, device=DEV)


def _dims(c, B, cap, pages, table, P=0):
    return dict(B=B, Hq=c["Hq"], Hkv=c["Hkv"], d=c["d"], bs=c["bs"], cap_tokens=cap, K=32, P=P, pages=pages,
                block_table=None if table is None else table.data_ptr())


def _finish(s, rows):
    """What a program of the library holds besides its tensors: its dims, and a workspace."""
    if own:
        import dynamic_sparse_attention_block_b200 as prr
        dims = prr.Dims(**s["dims"]).c()
        ws = torch.zeros(prr.prr_serving_workspace_bytes(dims, rows), dtype=torch.uint8, device=DEV)
        s.update(prr=prr, cdims=dims, ws=ws)
    return s


def _caches(c, g, B, cap, paged, lens, seed):
    """Caches in random order of pages, and the table; `lens`: what each sequence holds pages for."""
    Hkv, d, bs = c["Hkv"], c["d"], c["bs"]
    maxnb = _up(cap, bs)
    if not paged:
        return _randn(g, B, Hkv, cap, d), _randn(g, B, Hkv, cap, d), None, 0
    held = [_up(n, bs) for n in lens]
    pages = sum(held) + 3
    order = np.random.RandomState(seed % (1 << 31)).permutation(pages)
    table = np.full((B, maxnb), -1, np.int32)
    at = 0
    for b in range(B):
        table[b, :held[b]] = order[at:at + held[b]]
        at += held[b]
    return _randn(g, pages, Hkv, bs, d), _randn(g, pages, Hkv, bs, d), _i32(table), pages


def prepare(case, seed):
    c, g = case, _gen(seed)
    Hq, Hkv, d, bs = c["Hq"], c["Hkv"], c["d"], c["bs"]
    s = {"case": c}
    if c["op"] in ("append", "prompt"):
        new, old = _lengths(c)
        ends = [a + b for a, b in zip(new, old)]
        cap, B, T = max(ends), c["B"], sum(new)
        kc, vc, table, pages = _caches(c, g, B, cap, c["paged"], ends, seed)
        s.update(kc=kc, vc=vc, table=table, q_begin=_i32(np.concatenate([[0], np.cumsum(new)])), new=new, old=old,
                 dims=_dims(c, B, cap, pages, table), nb=_up(cap, bs))
        if c["op"] == "append":
            # the rows are parts of one projection's output, as they are in a model
            qkv = _randn(g, T, Hq + 2 * Hkv, d)
            s.update(k=qkv[:, Hq:Hq + Hkv], v=qkv[:, Hq + Hkv:], old_lens=_i32(old), lens=_i32(old))
            summ = torch.zeros(B, Hkv, s["nb"], 2, d, dtype=torch.bfloat16, device=DEV)
            for b in range(B):  # summaries of what is cached already
                if old[b]:
                    x = _seq(s, b, old[b], kc)
                    full = torch.nn.functional.pad(x, (0, 0, 0, _up(old[b], bs) * bs - old[b]), mode="replicate")
                    full = full.view(Hkv, -1, bs, d)
                    summ[b, :, :full.shape[1], 0], summ[b, :, :full.shape[1], 1] = full.amin(2), full.amax(2)
            s.update(summ=summ)
        else:
            s.update(q=_randn(g, T, Hq, d), lens=_i32(ends), out=torch.zeros(T, Hq, d, dtype=torch.bfloat16, device=DEV),
                     lse=torch.zeros(T, Hq, device=DEV))
        return _finish(s, T)
    if c["op"] == "shared":
        B, ng, pre = c["B"], c["groups"], c["prefix"]
        own_n = _own_lengths(c)
        n = [pre + x for x in own_n]
        cap = max(n)
        maxnb, pb, per = _up(cap, bs), pre // bs, B // ng
        if c["paged"]:
            tails = [_up(x, bs) for x in own_n]
            pages = ng * pb + sum(tails) + 3
            order = np.random.RandomState(seed % (1 << 31)).permutation(pages)
            t, at = np.full((B, maxnb), -1, np.int32), ng * pb
            for b in range(B):
                t[b, :pb] = order[(b % ng) * pb:(b % ng + 1) * pb]
                t[b, pb:pb + tails[b]] = order[at:at + tails[b]]
                at += tails[b]
            table, kc, vc = _i32(t), _randn(g, pages, Hkv, bs, d), _randn(g, pages, Hkv, bs, d)
        else:
            table, pages = None, 0
            kc, vc = _randn(g, B, Hkv, cap, d), _randn(g, B, Hkv, cap, d)
            for b in range(ng, B):
                kc[b, :, :pre], vc[b, :, :pre] = kc[b % ng, :, :pre], vc[b % ng, :, :pre]
        members = [b for i in range(ng) for b in range(i, B, ng)]  # slots of a batch are in no order
        s.update(kc=kc, vc=vc, table=table, q=_randn(g, B, Hq, d), lens=_i32(n), n=n, members=_i32(members), who=members,
                 group_begin=_i32(np.arange(ng + 1) * per), shared_blocks=_i32([pb] * ng), nb=maxnb,
                 out=torch.zeros(B, Hq, d, dtype=torch.bfloat16, device=DEV), lse=torch.zeros(B, Hq, device=DEV),
                 dims=_dims(c, B, cap, pages, table))
        return _finish(s, B)
    rs = np.random.RandomState(seed % (1 << 31))
    if c["op"] == "fork":
        ctx = _contexts(c)
        np_, nc = c["parents"], c["parents"] * c["children"]
        B, P = np_ + nc, 32
        cap = max(ctx) + bs
        maxnb = _up(cap, bs)
        held = [_up(n + 1, bs) for n in ctx]
        pages = sum(held) + 2 * nc + c["spare"]
        order = rs.permutation(pages)
        t, at, refs = np.full((B, maxnb), -1, np.int32), 0, np.zeros(pages, np.int32)
        for b in range(np_):
            t[b, :held[b]] = order[at:at + held[b]]
            at += held[b]
        refs[order[:at]] = 1
        lens = np.zeros(B, np.int32)
        lens[:np_] = ctx
        table = _i32(t)
        who = [i // c["children"] for i in range(nc)]
        s.update(table=table, refs=_i32(refs), lens=_i32(lens), parents=_i32(who), children=_i32(np_ + np.arange(nc)),
                 kc=_randn(g, pages, Hkv, bs, d), vc=_randn(g, pages, Hkv, bs, d),
                 summ=_randn(g, B, Hkv, maxnb, 2, d),
                 ema=torch.rand(B, Hkv, maxnb, dtype=torch.float64, device=DEV, generator=g),
                 pred=torch.randint(0, maxnb, (B, Hkv, P), dtype=torch.int32, device=DEV, generator=g),
                 tails=torch.tensor([i for i in range(nc) if ctx[who[i]] % bs], dtype=torch.int64, device=DEV),
                 want=torch.zeros(B, dtype=torch.int32, device=DEV), nb=maxnb, dims=_dims(c, B, cap, pages, table, P))
        return _finish(s, 1)
    # compact: sequences hold `live` pages of the pool, some of them shared by two
    B, pages, live = c["B"], c["pages"], c["live"]
    order = rs.permutation(pages)[:live]
    parts = np.array_split(order, B)
    maxnb = max(len(p) for p in parts) + 1
    t, refs = np.full((B, maxnb), -1, np.int32), np.zeros(pages, np.int32)
    for b in range(B):
        row = list(parts[b][:maxnb])
        if b and len(parts[b - 1]):
            row = [parts[b - 1][0]] + row  # the first page is also the neighbour's
        t[b, :len(row)] = row[:maxnb]
    np.add.at(refs, t[t >= 0], 1)
    table, moves = _i32(t), int((np.nonzero(refs)[0] >= (refs > 0).sum()).sum())
    s.update(table=table, table0=table.clone(), refs=_i32(refs), refs0=_i32(refs), moves=moves,
             remap=torch.zeros(pages, dtype=torch.int32, device=DEV), n_live=torch.zeros(1, dtype=torch.int32, device=DEV),
             kc=_randn(g, pages, Hkv, bs, d), vc=_randn(g, pages, Hkv, bs, d), nb=maxnb,
             dims=_dims(c, B, maxnb * bs, pages, table))
    return _finish(s, 1)


# ----------------------------------------------------------------------------- plain forms

def _seq(s, b, n, cache):
    """Tokens [0, n) of sequence b: [Hkv][n][d]."""
    bs = s["case"]["bs"]
    if s["table"] is None:
        return cache[b, :, :n]
    pages = s["table"][b, :_up(n, bs)].long()
    return cache[pages].transpose(0, 1).reshape(cache.shape[1], -1, cache.shape[3])[:, :n]


def _append(s):
    c = s["case"]
    bs, B, new, old = c["bs"], c["B"], s["new"], s["old"]
    T = sum(new)
    first = s["q_begin"][:-1].long()
    seq = torch.repeat_interleave(torch.arange(B, device=DEV), (s["q_begin"][1:] - s["q_begin"][:-1]).long(), output_size=T)
    pos = s["lens"].long()[seq] + torch.arange(T, device=DEV) - first[seq]
    if s["table"] is None:
        where = (seq, slice(None), pos)
    else:
        where = (s["table"][seq, pos // bs].long(), slice(None), pos % bs)
    s["kc"][where], s["vc"][where] = s["k"], s["v"]
    # the touched blocks, from their first token on
    spans = [(b, j, min(bs, old[b] + new[b] - j * bs)) for b in range(B)
             for j in range(old[b] // bs, _up(old[b] + new[b], bs))]
    sb, blk, valid = torch.tensor(spans, device=DEV).unbind(1)
    if s["table"] is None:
        tok = (blk[:, None] * bs + torch.arange(bs, device=DEV)).clamp(max=s["kc"].shape[2] - 1)
        rows = s["kc"][sb[:, None], :, tok].transpose(1, 2).float()
    else:
        rows = s["kc"][s["table"][sb, blk].long()].float()  # [touched][Hkv][bs][d]
    gone = (torch.arange(bs, device=DEV) >= valid[:, None])[:, None, :, None]
    s["summ"][sb, :, blk, 0] = rows.masked_fill(gone, math.inf).amin(2).bfloat16()
    s["summ"][sb, :, blk, 1] = rows.masked_fill(gone, -math.inf).amax(2).bfloat16()
    s["lens"] += s["q_begin"][1:] - s["q_begin"][:-1]


def _attend(q, k, v, scale, first):
    """q [rows][Hkv][G][d], k and v [Hkv][n][d]; row i sees tokens up to first + i (None: all). -> out, lse"""
    rows, Hkv, G, d = q.shape
    x = torch.matmul(q.permute(1, 2, 0, 3).reshape(Hkv, G * rows, d), k.transpose(1, 2)).mul_(scale)
    x = x.view(Hkv, G, rows, k.shape[1])
    if first is not None:
        x.masked_fill_(torch.arange(k.shape[1], device=DEV) > first + torch.arange(rows, device=DEV)[:, None], -math.inf)
    top = x.amax(-1, keepdim=True)
    x.sub_(top).exp_()
    total = x.sum(-1, keepdim=True)
    out = torch.matmul(x.view(Hkv, G * rows, -1), v).view(Hkv, G, rows, d) / total
    return out.permute(2, 0, 1, 3), (top + total.log())[..., 0].permute(2, 0, 1)


def _pieces(new, heads, ends):
    """Rows [i, j) of each sequence whose scores fit some gigabytes."""
    at = 0
    for b, rows in enumerate(new):
        step = max(1, min(rows, (1 << 30) // (heads * ends[b])))
        for i in range(0, rows, step):
            yield b, at, i, min(rows, i + step)
        at += rows


def _prompt(s, dtype=torch.float32):
    c = s["case"]
    Hq, Hkv, d = c["Hq"], c["Hkv"], c["d"]
    ends = [a + b for a, b in zip(s["new"], s["old"])]
    outs, lses, held, kv = [], [], -1, None
    for b, at, i, j in _pieces(s["new"], Hq, ends):
        if b != held:
            held, kv = b, [_seq(s, b, ends[b], x).to(dtype) for x in (s["kc"], s["vc"])]
        n = s["old"][b] + j
        o, l = _attend(s["q"][at + i:at + j].view(j - i, Hkv, Hq // Hkv, d).to(dtype), kv[0][:, :n], kv[1][:, :n],
                       1 / math.sqrt(d), s["old"][b] + i)
        outs.append(o.reshape(j - i, Hq, d).bfloat16() if dtype == torch.float32 else o.reshape(j - i, Hq, d))
        lses.append(l.reshape(j - i, Hq))
    return {"out": torch.cat(outs), "lse": torch.cat(lses)}


def _shared(s):
    c = s["case"]
    Hq, Hkv, d, bs, ng, pre = c["Hq"], c["Hkv"], c["d"], c["bs"], c["groups"], c["prefix"]
    G, scale, m = Hq // Hkv, 1 / math.sqrt(d), s["members"].long()
    q = s["q"][m].float().view(ng, -1, Hkv, G, d).permute(0, 2, 1, 3, 4)  # [groups][Hkv][members][G][d]
    per = q.shape[2]
    # the members' own tokens, padded to the longest
    longest = max(s["n"]) - pre
    tok = pre + torch.arange(longest, device=DEV)
    if s["table"] is None:
        kv = [x[m][:, :, pre:pre + longest].float() for x in (s["kc"], s["vc"])]
    else:
        page = s["table"][m][:, tok // bs].clamp(min=0).long()
        kv = [x[page, :, (tok % bs)[None]].transpose(1, 2).float() for x in (s["kc"], s["vc"])]
    own_x = torch.matmul(q.transpose(1, 2).reshape(ng * per, Hkv, G, d), kv[0].transpose(2, 3)) * scale
    gone = tok >= s["lens"].long()[m][:, None]
    own_x.masked_fill_(gone[:, None, None], -math.inf)
    own_v = kv[1].masked_fill(gone[:, None, :, None], 0)
    out, lse = torch.empty_like(s["out"]), torch.empty_like(s["lse"])
    for i in range(ng):
        k, v = (_seq(s, s["who"][i * per], pre, x).float() for x in (s["kc"], s["vc"]))
        x = torch.matmul(q[i].reshape(Hkv, per * G, d), k.transpose(1, 2)).mul_(scale).view(Hkv, per, G, pre)
        y = own_x[i * per:(i + 1) * per].transpose(0, 1)
        top = torch.maximum(x.amax(-1, keepdim=True), y.amax(-1, keepdim=True))
        x, y = x.sub_(top).exp_(), (y - top).exp()
        total = x.sum(-1, keepdim=True) + y.sum(-1, keepdim=True)
        o = torch.matmul(x.view(Hkv, per * G, pre), v).view(Hkv, per, G, d)
        o = (o + torch.matmul(y, own_v[i * per:(i + 1) * per].transpose(0, 1))) / total
        rows = m[i * per:(i + 1) * per]
        out[rows] = o.transpose(0, 1).reshape(per, Hq, d).bfloat16()
        lse[rows] = (top + total.log())[..., 0].transpose(0, 1).reshape(per, Hq)
    return {"out": out, "lse": lse}


def _free_pages(s):
    """Page numbers, the free ones first, in ascending order."""
    return torch.argsort((s["refs"] > 0).to(torch.uint8), stable=True)


def _fork(s):
    table, refs, lens = s["table"], s["refs"], s["lens"]
    kids, pars, bs = s["children"].long(), s["parents"].long(), s["case"]["bs"]
    # release the children
    rows = table[kids]
    refs.index_add_(0, rows.clamp(min=0).reshape(-1).long(), -(rows >= 0).to(torch.int32).reshape(-1))
    table[kids], lens[kids] = -1, 0
    # fork the parents: whole pages are shared, the last one, where it is not full, is copied
    n = lens[pars]
    full, blocks = n // bs, (n + bs - 1) // bs
    j = torch.arange(s["nb"], device=DEV)
    held = j < full[:, None]
    rows = torch.where(held, table[pars], -1)
    refs.index_add_(0, rows.clamp(min=0).reshape(-1).long(), held.to(torch.int32).reshape(-1))
    table[kids] = rows
    t = s["tails"]
    last = full[t].long()
    src, dst = table[pars[t], last].long(), _free_pages(s)[:t.numel()]
    table[kids[t], last] = dst.to(torch.int32)
    refs[dst] = 1
    s["kc"][dst], s["vc"][dst] = s["kc"][src], s["vc"][src]
    seen = j < blocks[:, None]
    s["summ"][kids] = torch.where(seen[:, None, :, None, None], s["summ"][pars], s["summ"][kids])
    s["ema"][kids] = torch.where(seen[:, None], s["ema"][pars], 0.0)
    s["pred"][kids] = s["pred"][pars]
    lens[kids] = n
    # room for the next token of every sequence
    s["want"].copy_(lens + 1)
    missing = (j < ((s["want"] + bs - 1) // bs)[:, None]) & (table < 0)
    rank = (missing.reshape(-1).cumsum(0) - 1).clamp(0, refs.numel() - 1).view_as(table)
    page = _free_pages(s)[rank]
    refs.index_add_(0, page.reshape(-1), missing.to(torch.int32).reshape(-1))
    table.copy_(torch.where(missing, page.to(torch.int32), table))


def _compact(s):
    refs, i = s["refs"], torch.arange(s["refs"].numel(), device=DEV)
    live = refs > 0
    n = live.sum()
    mover = live & (i >= n)
    to = _free_pages(s)[(mover.cumsum(0) - 1).clamp(min=0)]
    remap = torch.where(mover, to, torch.where(live, i, -1))
    src = torch.argsort((~mover).to(torch.uint8), stable=True)[:s["moves"]]
    dst = remap[src]
    s["kc"][dst], s["vc"][dst] = s["kc"][src], s["vc"][src]
    refs[dst] = refs[src]
    refs[src] = 0
    s["remap"].copy_(remap)
    s["n_live"].copy_(n)
    t = s["table"]
    t.copy_(torch.where(t >= 0, s["remap"][t.clamp(min=0).long()], t))


# ----------------------------------------------------------------------------- one pass

def _buffers(s):
    return s["prr"].cache_buffers(k_cache=s["kc"], v_cache=s["vc"], block_table=s["table"], page_refs=s["refs"],
                                  seq_lens=s.get("lens"), summ=s.get("summ"), ema=s.get("ema"), pred=s.get("pred"))


def run(state):
    s = state
    op = s["case"]["op"]
    if op == "append":
        s["lens"].copy_(s["old_lens"])
        if own:
            s["prr"].prr_append_prompt(s["cdims"], s["k"], s["v"], s["q_begin"], s["lens"], s["kc"], s["vc"], s["summ"],
                                       s["ws"])
        else:
            _append(s)
        return {"k_cache": s["kc"], "v_cache": s["vc"], "summ": s["summ"], "seq_lens": s["lens"]}
    if op == "prompt":
        if own:
            s["prr"].prr_attend_prompt(s["cdims"], s["q"], s["q_begin"], s["lens"], s["kc"], s["vc"], s["out"], s["lse"],
                                       s["ws"])
            return {"out": s["out"], "lse": s["lse"]}
        return _prompt(s)
    if op == "shared":
        if own:
            s["prr"].prr_attend_shared(s["cdims"], s["q"], s["members"], s["group_begin"], s["shared_blocks"], s["lens"],
                                       s["kc"], s["vc"], s["out"], s["lse"], s["ws"])
            return {"out": s["out"], "lse": s["lse"]}
        return _shared(s)
    if op == "fork":
        if own:
            prr, dims, ws, bufs = s["prr"], s["cdims"], s["ws"], _buffers(s)
            prr.prr_cache_release(dims, s["children"], bufs, ws)
            prr.prr_cache_fork(dims, s["parents"], s["children"], bufs, ws)
            torch.add(s["lens"], 1, out=s["want"])
            prr.prr_cache_reserve(dims, s["want"], bufs, ws)
        else:
            _fork(s)
        return {k: s[k] for k in ("table", "refs", "lens", "kc", "vc", "summ", "ema", "pred")}
    s["table"].copy_(s["table0"])
    s["refs"].copy_(s["refs0"])
    if own:
        s["prr"].prr_cache_compact(s["cdims"], _buffers(s), s["remap"], s["n_live"], s["ws"])
    else:
        _compact(s)
    return {k: s[k] for k in ("table", "refs", "remap", "n_live", "kc", "vc")}


def work(case):
    c = case
    Hq, Hkv, d, bs = c["Hq"], c["Hkv"], c["d"], c["bs"]
    row = 2 * Hkv * d * 2  # K and V of one token
    if c["op"] in ("append", "prompt"):
        new, old = _lengths(c)
        T = sum(new)
        if c["op"] == "append":
            blocks = sum(_up(a + b, bs) - b // bs for a, b in zip(new, old))
            return {"bytes": 2 * T * row + blocks * Hkv * 2 * d * 2, "flops": 2 * T * Hkv * d}
        pairs = sum(a * b + a * (a + 1) // 2 for a, b in zip(new, old))
        return {"bytes": T * Hq * (4 * d + 4) + sum(a + b for a, b in zip(new, old)) * row, "flops": 4 * d * Hq * pairs}
    if c["op"] == "shared":
        own_n = _own_lengths(c)
        tokens = c["groups"] * c["prefix"] + sum(own_n)
        return {"bytes": tokens * row + c["B"] * Hq * (4 * d + 4),
                "flops": 4 * d * Hq * (c["B"] * c["prefix"] + sum(own_n))}
    if c["op"] == "fork":
        per = [2 * (row * bs * (n % bs > 0) + _up(n, bs) * Hkv * (4 * d + 8) + 32 * Hkv * 4) for n in _contexts(c)]
        return {"bytes": c["children"] * sum(per), "flops": 0}
    # a live page stands behind the live count with the chance of a free one
    moved = c["live"] * (c["pages"] - c["live"]) / c["pages"]
    return {"bytes": 2 * moved * row * bs + 2 * 4 * c["pages"], "flops": 0}


# ----------------------------------------------------------------------------- in 64 bits

def exact(case, seed):
    """Attention straight from its definition, one sequence at a time. The other operators move values and compute
    none."""
    c = case
    if c["op"] not in ("prompt", "shared"):
        return None
    if work(c)["flops"] > 3e13:
        return None
    s = prepare(c, seed)
    Hq, Hkv, d, bs = c["Hq"], c["Hkv"], c["d"], c["bs"]
    if c["op"] == "prompt":
        new, old = _lengths(c)
        ask = [(b, i) for b in range(c["B"]) for i in range(new[b])]
        spans = [(b, sum(new[:b]), i, min(new[b], i + 512)) for b in range(c["B"]) for i in range(0, new[b], 512)]
    else:
        new = old = None
        ask = [(b, 0) for b in range(c["B"])]
        spans = [(b, b, 0, 1) for b in range(c["B"])]
    out = torch.empty(len(ask), Hq, d, dtype=torch.float64, device=DEV)
    lse = torch.empty(len(ask), Hq, dtype=torch.float64, device=DEV)
    held, k, v = -1, None, None
    for b, at, i, j in spans:
        n = old[b] + new[b] if new else s["n"][b]
        if b != held:
            held = b
            if s["table"] is None:
                k, v = s["kc"][b, :, :n], s["vc"][b, :, :n]
            else:
                page, off = s["table"][b].long()[torch.arange(n, device=DEV) // bs], torch.arange(n, device=DEV) % bs
                k, v = (x[page, :, off].transpose(0, 1) for x in (s["kc"], s["vc"]))
            k, v = k.double(), v.double()
        sees = torch.arange(n, device=DEV) <= (old[b] + torch.arange(i, j, device=DEV) if new else
                                               torch.full((1,), n - 1, device=DEV))[:, None]
        for h in range(Hq):
            logits = s["q"][at + i:at + j, h].double() @ k[h * Hkv // Hq].T / math.sqrt(d)
            logits = torch.where(sees, logits, -math.inf)
            lse[at + i:at + j, h] = torch.logsumexp(logits, -1)
            out[at + i:at + j, h] = torch.exp(logits - lse[at + i:at + j, h, None]) @ v[h * Hkv // Hq]
    return {"out": out, "lse": lse}
