"""What the calls around the decode step leave behind for the steps that follow: empty and
released slots, queries that are not finite, checkpoints, workspaces of captured calls.
Needs a B200; marked gpu."""
import math

import numpy as np
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():  # collected on CPU-only machines, never run there
    pytest.skip("needs a CUDA GPU", allow_module_level=True)

import dynamic_sparse_attention_block_b200 as prr  # noqa: E402
from tests.test_gpu_serving import Case, _i32, _prompt, _shared, _some  # noqa: E402

DEV = "cuda"
NAN, INF = float("nan"), float("inf")


def _tokens(n, *heads, d, seed=0):
    g = torch.Generator(device=DEV).manual_seed(seed)
    return [torch.randn(n, h, d, generator=g, device=DEV).bfloat16() for h in heads]


def _step(dec, mode, q, k=None, v=None):
    """One decode step; k, v: the token it appends ("host": appended by a call of its own before it)."""
    if mode == "fused":
        dec.step_fused(q, k_new=k, v_new=v)
    elif mode == "host":
        if k is not None:
            dec.append(k, v)
        dec.step_fused(q)
    else:
        if k is not None:
            dec.k_new.copy_(k)
            dec.v_new.copy_(v)
        dec.step(q, append=k is not None)
    torch.cuda.synchronize()


# ----------------------------------------------------------------------------- predictions

@pytest.mark.parametrize("mode", ["fused", "streams"])
@pytest.mark.parametrize("released", [False, True])
@pytest.mark.parametrize("n,P,cap", [(1, 8, 1024), (10, 64, 1024), (64, 2, 1024), (200, 7, 256), (900, 15, 1024)])
def test_a_prompt_shorter_than_the_prediction_in_an_empty_slot(n, P, cap, released, mode):
    """A fresh or released slot predicts as the zero state does at the length that its prompt gives it: the step
    equals that of a decoder that was prefilled, and reports nothing."""
    Hq, Hkv, d, bs = 8, 2, 64, 64
    sizes = dict(B=1, Hq=Hq, Hkv=Hkv, d=d, bs=bs, cap_tokens=cap, K=4, P=P)
    dec = prr.PRRDecoder(prr.Dims(pages=40, **sizes), empty=True)
    k, v, q = _tokens(n, Hkv, Hkv, Hq, d=d)
    if released:
        k0, v0, q0 = _tokens(250, Hkv, Hkv, Hq, d=d, seed=1)
        dec.reserve([251])
        dec.append_prompt(k0, v0, [0, 250])
        _step(dec, mode, q0[:1])
        dec.release([0])
    dec.reserve([n])
    dec.append_prompt(k, v, [0, n])
    flat = prr.PRRDecoder(prr.Dims(**sizes))
    flat.prefill(k.transpose(0, 1)[None], v.transpose(0, 1)[None], n)
    for x in (dec, flat):
        _step(x, mode, q[-1:])
    assert flat.device_status() == 0 and dec.device_status() == 0
    for name in ("sel", "missed", "n_missed", "keep", "pred"):
        a, b = getattr(dec, name), getattr(flat, name)
        if name == "missed":  # entries past the count are left as they were
            m = int(dec.n_missed.max())
            a, b = a[..., :m], b[..., :m]
        assert torch.equal(a, b), name
    assert (dec.out - flat.out).abs().max() < 1e-5 and (dec.lse - flat.lse).abs().max() < 1e-5


@pytest.mark.parametrize("entries", [[4, -1, -1], [0, 4, -1], [-2, -1, -1], [1, 0, -1], [0, 1, 3]])
def test_a_prediction_of_blocks_that_are_not_there_is_still_reported(entries):
    n, Hkv, Hq, d = 130, 1, 2, 64  # three blocks of a cache of sixteen
    dec = prr.PRRDecoder(prr.Dims(B=1, Hq=Hq, Hkv=Hkv, d=d, bs=64, cap_tokens=1024, K=2, P=3))
    k, v, q = _tokens(n, Hkv, Hkv, Hq, d=d)
    dec.prefill(k.transpose(0, 1)[None], v.transpose(0, 1)[None], n)
    dec.pred.copy_(_i32([[entries]]))
    _step(dec, "fused", q[-1:])
    assert dec.device_status() == 2


# ----------------------------------------------------------------------------- queries that are not finite

def _spoil(q, rows):
    """Every third of the rows gets one head that holds a NaN or an infinity; returns {row: head}."""
    bad = {}
    for i, r in enumerate(rows[::3]):
        h = (5 * i) % q.shape[1]
        q[r, h, i % q.shape[2]] = (NAN, INF, -INF)[i % 3]
        bad[r] = h
    return bad


def _check_spoiled(c, q, bad, out, lse, rows):
    clean = q.clone()
    for r, h in bad.items():
        clean[r, h] = 0
    o, l = out.clone(), lse.clone()
    for r, b, n in rows:
        if r in bad:  # one head of the row: NaN in every channel; the others as they are
            h = bad[r]
            assert bool(out[r, h].isnan().all()), (r, b, n, out[r, h][:4])
            assert not bool(lse[r, h].isfinite()), (r, b, n)
            if bool(q[r, h].isnan().any()):
                assert bool(lse[r, h].isnan()), (r, b, n)
            eo, el, _, _ = c.exact(clean[r], b, n)
            o[r, h], l[r, h] = eo[h], el[h].float()
    c.check(clean, o, l, rows)


@pytest.mark.parametrize("Hq,Hkv,d,bs,paged,new,old", [
    (32, 8, 128, 64, True, [300], [0]),         # whole and cut tiles of more than 128 rows
    (4, 1, 64, 64, False, [3], [20000]),        # few rows, cut between all CTAs
    (8, 2, 128, 128, True, [1] * 400, [70] * 400),  # one piece a sequence, of few rows
    (6, 2, 64, 64, True, [40, 1, 130], [500, 0, 9000]),
])
def test_attend_prompt_queries_that_are_not_finite(Hq, Hkv, d, bs, paged, new, old):
    c = Case(Hq, Hkv, d, bs, [a + b for a, b in zip(new, old)], paged)
    q = c.randn(sum(new), Hq, d)
    at = np.concatenate([[0], np.cumsum(new)])
    rows = _some([(int(at[b]) + i, b, old[b] + i + 1) for b in range(c.B) for i in range(new[b])], 60)
    bad = _spoil(q, [r for r, _, _ in rows])
    q, _, out, lse, ws = _prompt(c, new, q=q)
    _check_spoiled(c, q, bad, out, lse, rows)
    assert prr.prr_get_device_status(ws) == 0


@pytest.mark.parametrize("prefix,own", [([20, 0], [[5, 600, 0, 129], [1, 77, 0]]), ([300], [[1] * 70]), ([0], [[9000]])])
def test_attend_shared_queries_that_are_not_finite(prefix, own):
    bs, lens, gb, share = 64, [], [0], []
    for pb, tails in zip(prefix, own):
        first = len(lens)
        lens += [pb * bs + t for t in tails]
        share += [(first, b, pb * bs) for b in range(first + 1, len(lens))]
        gb.append(len(lens))
    c = Case(8, 2, 128, bs, lens, True, share=share)
    q = c.randn(c.B, 8, 128)
    bad = _spoil(q, list(range(c.B)))
    q[[b for b in range(c.B) if lens[b] == 0]] = NAN
    q, out, lse, ws = _shared(c, list(range(c.B)), gb, prefix, q=q)
    _check_spoiled(c, q, bad, out, lse, [(b, b, lens[b]) for b in range(c.B) if lens[b]])
    for b in range(c.B):
        if lens[b] == 0:  # attends nothing, whatever its query
            assert bool((out[b] == 0).all()) and bool((lse[b] == -math.inf).all())
    assert prr.prr_get_device_status(ws) == 0


# ----------------------------------------------------------------------------- checkpoints, the caller's tensors

def _representative(seed=0):
    B, Hq, Hkv, d, bs, n_rep = 2, 4, 2, 64, 64, 2
    g = torch.Generator().manual_seed(seed)
    dims = prr.Dims(B=B, Hq=Hq, Hkv=Hkv, d=d, bs=bs, cap_tokens=1024, K=3, P=2, pages=40, selector="representative",
                    n_rep=n_rep)
    rep = torch.randint(0, bs, (B, Hkv, dims.maxnb, n_rep), generator=g, dtype=torch.uint8)
    return dims, rep


def test_a_checkpoint_holds_the_representatives_that_a_fork_copied():
    n = 900
    dims, rep = _representative()
    k, v, q = _tokens(n, 2, 2, 4, d=64)
    kn, vn, qn = _tokens(2, 2, 2, 4, d=64, seed=3)
    dec = prr.PRRDecoder(dims, rep_offsets=rep, empty=True)
    dec.reserve([n, 0])
    dec.append_prompt(k, v, [0, n, n])
    before = dec.checkpoint()
    dec.fork([0], [1])
    dec.reserve([n + 2] * 2)
    ck = dec.checkpoint()
    other = prr.PRRDecoder(dims, rep_offsets=rep, empty=True)
    other.restore(ck)
    for x in (dec, other):
        _step(x, "fused", qn, kn, vn)
    assert torch.equal(other.rep_offsets, dec.rep_offsets)
    assert torch.equal(other.sel, dec.sel) and torch.equal(other.out, dec.out)
    dec.restore(before)  # back across the fork
    assert torch.equal(dec.rep_offsets.cpu(), rep)
    del ck["rep_offsets"]  # of a decoder that never forked: the offsets it was built with are its own
    other.restore(ck)
    assert other.device_status() == 0


def test_the_callers_table_and_offsets_are_not_written():
    dims, rep = _representative(1)
    table = torch.full((2, dims.maxnb), -1, dtype=torch.int32, device=DEV)
    table[0, :3] = _i32([7, 1, 30])
    rep = rep.to(DEV)
    rep0, table0 = rep.clone(), table.clone()
    dec = prr.PRRDecoder(dims, block_table=table, rep_offsets=rep)
    dec.seq_lens.copy_(_i32([150, 0]))
    dec.fork([0], [1])
    dec.compact()
    dec.reserve([150, 400])
    dec.release([0])
    assert dec.device_status() == 0 and not torch.equal(dec.block_table, table0)
    assert torch.equal(dec.rep_offsets[1, :, :3], rep0[0, :, :3])
    assert torch.equal(table, table0) and torch.equal(rep, rep0)


# ----------------------------------------------------------------------------- slots without tokens, tokens without pages

@pytest.mark.parametrize("mode", ["fused", "host", "streams"])
@pytest.mark.parametrize("selector", ["group_sum", "per_head"])
def test_steps_pass_over_slots_that_hold_nothing(mode, selector):
    """A batch with idle slots decodes as the others alone would; the idle ones can be filled and forked into after."""
    Hq, Hkv, d, bs, n = 8, 2, 64, 64, 300
    sizes = dict(Hq=Hq, Hkv=Hkv, d=d, bs=bs, cap_tokens=1024, K=3, P=3, selector=selector)
    dec = prr.PRRDecoder(prr.Dims(B=4, pages=60, **sizes), empty=True)
    one = prr.PRRDecoder(prr.Dims(B=1, **sizes))
    k, v = _tokens(n, Hkv, Hkv, d=d)
    dec.reserve([50, n + 8, 0, 0])
    dec.append_prompt(torch.cat([k[:50], k]), torch.cat([v[:50], v]), [0, 50, 50 + n, 50 + n, 50 + n])
    dec.release([0])  # slot 0 was used, slots 2 and 3 never were
    one.prefill(k.transpose(0, 1)[None], v.transpose(0, 1)[None], n)
    idle = [0, 2, 3]
    for step in range(4):
        q, kn, vn = _tokens(4, Hq, Hkv, Hkv, d=d, seed=10 + step)
        token = (kn, vn) if step != 2 else (None, None)
        _step(dec, mode, q, *token)
        _step(one, mode, q[1:2], *(x if x is None else x[1:2] for x in token))
        assert dec.device_status() == 0 and one.device_status() == 0, step
        assert dec.seq_lens.tolist() == [0, int(one.seq_lens), 0, 0], step
        assert bool((dec.out[idle] == 0).all()) and bool((dec.lse[idle] == -INF).all()), step
        assert bool((dec.sel[idle] == -1).all()) and not bool(dec.n_missed[idle].any()) and not bool(dec.keep[idle].any())
        assert not bool(dec.ema[idle].any()) and bool((dec.block_table[idle] == -1).all()), step
        assert torch.equal(dec.sel[1], one.sel[0]) and torch.equal(dec.pred[1], one.pred[0]), step
        assert (dec.out[1] - one.out[0]).abs().max() < 1e-5, step
    now = int(one.seq_lens)
    dec.fork([1], [2])
    dec.reserve([n + 1, now + 1, now + 1, 0])
    dec.append_prompt(k, v, [0, n, n, n, n])
    q, kn, vn = _tokens(4, Hq, Hkv, Hkv, d=d, seed=20)
    q[2], kn[2], vn[2] = q[1], kn[1], vn[1]
    fresh = prr.PRRDecoder(prr.Dims(B=1, **sizes))
    fresh.prefill(k.transpose(0, 1)[None], v.transpose(0, 1)[None], n)
    _step(dec, mode, q, kn, vn)
    _step(one, mode, q[1:2], kn[1:2], vn[1:2])
    _step(fresh, mode, q[:1], kn[:1], vn[:1])
    assert dec.device_status() == 0 and dec.seq_lens.tolist() == [n + 1, now + 1, now + 1, 0]
    for b, x in ((0, fresh), (1, one), (2, one)):
        assert torch.equal(dec.sel[b], x.sel[0]) and (dec.out[b] - x.out[0]).abs().max() < 1e-5, b
    assert bool((dec.out[3] == 0).all()) and bool((dec.lse[3] == -INF).all())


@pytest.mark.parametrize("mode", ["fused", "host", "streams"])
def test_a_step_starts_an_empty_sequence_that_has_its_page(mode):
    dec = prr.PRRDecoder(prr.Dims(B=3, Hq=4, Hkv=1, d=64, bs=64, cap_tokens=256, K=4, P=2, pages=9), empty=True)
    dec.reserve([0, 1, 70])
    q, k, v = _tokens(3, 4, 1, 1, d=64)
    _step(dec, mode, q, k, v)
    assert dec.device_status() == 0 and dec.seq_lens.tolist() == [0, 1, 1]
    assert torch.equal(dec.out[1:], v[1:].float().expand(2, 4, 64)) and bool((dec.out[0] == 0).all())
    assert torch.equal(dec.summ[1:, :, 0, 0], k[1:]) and torch.equal(dec.summ[1:, :, 0, 1], k[1:])


def test_separate_calls_pass_over_an_empty_slot_and_report_an_empty_sequence_of_a_contiguous_cache():
    dims = prr.Dims(B=2, Hq=4, Hkv=1, d=64, bs=64, cap_tokens=256, K=4, P=2, pages=9)
    dec = prr.PRRDecoder(dims, empty=True)
    dec.reserve([0, 5])
    q, k, v = _tokens(2, 4, 1, 1, d=64)
    dec.append(k, v)
    prr.prr_update_summaries(dec.dims, dec.k_cache, None, None, dec.seq_lens, 1, dec.summ, dec.ws, dec.select_stream)
    dec.select_stream.synchronize()
    assert dec.device_status() == 0 and dec.seq_lens.tolist() == [0, 1] and torch.equal(dec.summ[1, 0, 0, 0], k[1, 0])
    flat = prr.PRRDecoder(prr.Dims(B=2, Hq=4, Hkv=1, d=64, bs=64, cap_tokens=256, K=4, P=2))
    _step(flat, "fused", q)
    assert flat.device_status() == 1


@pytest.mark.parametrize("mode", ["fused", "host", "streams"])
@pytest.mark.parametrize("n,entry", [(64, -1), (128, 10 ** 6), (70, -1)])
def test_a_token_without_a_page_is_dropped_and_can_be_given_again(mode, n, entry):
    """Its sequence keeps its length, so that reserve() still sees the missing block and the next step appends there."""
    dims = prr.Dims(B=2, Hq=4, Hkv=2, d=64, bs=64, cap_tokens=512, K=8, P=2, pages=12)
    dec = prr.PRRDecoder(dims, empty=True)
    k, v = _tokens(n, 2, 2, d=64)
    dec.reserve([n, n + 2])
    dec.append_prompt(torch.cat([k, k]), torch.cat([v, v]), [0, n, 2 * n])
    page = int(dec.block_table[0, n // 64])
    dec.block_table[0, n // 64] = entry
    q, kn, vn = _tokens(2, 4, 2, 2, d=64, seed=2)
    _step(dec, mode, q, kn, vn)
    assert dec.device_status() == 5 and dec.seq_lens.tolist() == [n, n + 1]
    prr.prr_workspace_init(dec.ws)
    dec.block_table[0, n // 64] = page
    dec.reserve([n + 1, n + 2])
    q[1], kn[1], vn[1] = q[0], kn[0], vn[0]
    _step(dec, mode, q, kn, vn)
    assert dec.device_status() == 0 and dec.seq_lens.tolist() == [n + 1, n + 2]
    kk, vv = (torch.cat([x, y[:1]]).double().repeat_interleave(2, 1) for x, y in ((k, kn), (v, vn)))
    w = torch.softmax(torch.einsum("hd,nhd->hn", q[0].double(), kk) / 8, -1)
    # weights in two bf16 parts (2^-16 of each), fp32 sums
    assert (dec.out[0] - torch.einsum("hn,nhd->hd", w, vv)).abs().max() < 2.0 ** -13


# ----------------------------------------------------------------------------- captured calls

def test_a_captured_call_keeps_its_workspace_when_a_later_call_needs_a_larger_one():
    Hq, Hkv, d, n, small = 8, 2, 64, 6000, 40
    dec = prr.PRRDecoder(prr.Dims(B=1, Hq=Hq, Hkv=Hkv, d=d, bs=64, cap_tokens=n, K=4, P=0, pages=100), empty=True)
    c = Case(Hq, Hkv, d, 64, [n], False)
    k, v = (x[0].transpose(0, 1).contiguous() for x in (c.k, c.v))
    q = c.randn(n, Hq, d)
    dec.reserve([n])
    dec.append_prompt(k[:small], v[:small], [0, small])
    qb, qs = _i32([0, small]), q[:small].contiguous()
    want, want_lse = dec.attend_prompt(qs, qb)
    torch.cuda.synchronize()
    used = dec.serve_ws.numel()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out, lse = dec.attend_prompt(qs, qb)
    dec.append_prompt(k[small:], v[small:], [0, n - small])
    assert dec.serve_ws.numel() == used  # appended rows take no room there
    o, l = dec.attend_prompt(q, [0, n])
    assert dec.serve_ws.numel() > used
    c.check(q, o, l, _some((i, 0, i + 1) for i in range(n)))
    with torch.cuda.stream(dec.select_stream):  # whatever was given back is in use again
        junk = [torch.full((used,), 171, dtype=torch.uint8, device=DEV) for _ in range(4)]
    torch.cuda.synchronize()
    dec.seq_lens.fill_(small)
    torch.cuda.synchronize()
    for _ in range(2):
        out.zero_()
        lse.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want) and torch.equal(lse, want_lse)
    assert all(bool((x == 171).all()) for x in junk)
    assert dec.device_status() == 0
    dec.seq_lens.fill_(small - 1)  # fewer tokens than rows: the replay's own status is read too
    graph.replay()
    torch.cuda.synchronize()
    assert dec.device_status() == 1


def test_load_context_needs_the_pages_it_writes():
    dec = prr.PRRDecoder(prr.Dims(B=2, Hq=4, Hkv=1, d=64, bs=64, cap_tokens=512, K=4, P=0, pages=6), empty=True)
    k, v = _tokens(130, 1, 1, d=64)
    dec.reserve([0, 64])
    for n in (1, 65, 130):
        for b in (0, 1):
            if (b, n) != (1, 1):
                with pytest.raises(ValueError, match="reserve"):
                    dec.load_context(b, 0, k[:n, 0], v[:n, 0])
    assert not bool(dec.k_cache.any()) and not bool(dec.v_cache.any())
    dec.reserve([130, 0])
    dec.load_context(0, 0, k[:, 0], v[:, 0])
    pages = dec.block_table[0, :3].long()
    assert torch.equal(dec.k_cache[pages, 0].reshape(-1, 64)[:130], k[:, 0])
    dec.block_table[0, 1] = 6  # past the pool
    with pytest.raises(ValueError, match="reserve"):
        dec.load_context(0, 0, k[:, 0], v[:, 0])


# ----------------------------------------------------------------------------- forks in one call

@pytest.mark.parametrize("parents,children,done", [
    ([0, 1], [2, 3], {2: 0, 3: 1}),
    ([0, 1], [1, 2], {}),           # 1 is not empty, and as a child of the call no parent either
    ([0, 2], [2, 3], {2: 0}),       # a chain: 2 becomes a copy of 0, 3 gets nothing
    ([2, 0], [3, 2], {2: 0}),       # in the other order too
    ([0, 0], [0, 2], {}),           # its own child
    ([2, 0], [3, 4], {3: 2, 4: 0}),  # a copy of an empty sequence is empty
])
def test_fork_entries_that_name_each_other(parents, children, done):
    lens = [100, 64, 0, 0, 0]
    table, refs = _i32([[3, 1], [5, -1], [-1, -1], [-1, -1], [-1, -1]]), _i32([0, 1, 0, 1, 0, 1, 0, 0])
    dims = prr.Dims(B=5, Hq=1, Hkv=1, d=64, bs=64, cap_tokens=128, K=1, P=0, pages=8, block_table=table.data_ptr())
    kc = torch.arange(8, device=DEV).view(8, 1, 1, 1).expand(8, 1, 64, 64).bfloat16().contiguous()
    vc, n = kc.clone(), _i32(lens)
    ws = torch.zeros(prr.prr_serving_workspace_bytes(dims, 1), dtype=torch.uint8, device=DEV)
    want, free, held = table.tolist(), iter([0, 2, 4]), refs.tolist()
    for p, c in zip(parents, children):
        if done.get(c) == p:
            lens[c] = lens[p]
            for j in range(lens[p] // 64):
                want[c][j] = want[p][j]
                held[want[p][j]] += 1
            if lens[p] % 64:
                want[c][lens[p] // 64] = pg = next(free)
                held[pg] = 1
    prr.prr_cache_fork(dims, _i32(parents), _i32(children), prr.cache_buffers(kc, vc, table, refs, n), ws)
    assert prr.prr_get_device_status(ws) == (0 if len(done) == len(children) else 5)
    assert table.tolist() == want and refs.tolist() == held and n.tolist() == lens


# ----------------------------------------------------------------------------- reservations past 32 bits

def test_a_reservation_of_more_blocks_than_32_bits_count_changes_nothing():
    B, bs, cap = 128, 64, 1 << 30  # 2^31 blocks are asked for: as 32 bits, a negative number
    table = torch.full((B, cap // bs), -1, dtype=torch.int32, device=DEV)
    refs, lens = _i32([0, 1, 0, 0]), _i32([0] * B)
    dims = prr.Dims(B=B, Hq=1, Hkv=1, d=64, bs=bs, cap_tokens=cap, K=1, P=0, pages=4, block_table=table.data_ptr())
    ws = torch.zeros(prr.prr_serving_workspace_bytes(dims, 1), dtype=torch.uint8, device=DEV)
    bufs = prr.cache_buffers(block_table=table, page_refs=refs, seq_lens=lens)
    prr.prr_cache_reserve(dims, _i32([cap] * B), bufs, ws)
    assert prr.prr_get_device_status(ws) == 6
    assert refs.tolist() == [0, 1, 0, 0] and int(table.max()) == -1
    prr.prr_workspace_init(ws)
    prr.prr_cache_reserve(dims, _i32([bs] * 3 + [0] * (B - 3)), bufs, ws)
    assert prr.prr_get_device_status(ws) == 0
    assert refs.tolist() == [1] * 4 and table[:4, :2].tolist() == [[0, -1], [2, -1], [3, -1], [-1, -1]]
