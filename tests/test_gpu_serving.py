"""The calls around the decode step -- packed prompts, shared prefixes, shared pages --
against plain 64-bit forms.  Needs a B200; marked gpu.

Tolerances of the attention outputs, per element and before any run: the weights are
rounded to bf16 once (half a step, 2^-8 of each) before the sum over v, and the result
once, so |out - exact| <= 2^-8 * (sum_j w_j |v_j| + |exact|), plus fp32 sums.  lse stays in fp32: a
logit is off by at most (d + 2) * 2^-24 * scale * sum_c |q_c k_c|, exponentials and
logarithms by 2^-21, and a running sum of n terms by n * 2^-24 relative.
"""
import math

import numpy as np
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():  # collected on CPU-only machines, never run there
    pytest.skip("needs a CUDA GPU", allow_module_level=True)

import dynamic_sparse_attention_block_b200 as prr  # noqa: E402

DEV = "cuda"
NAN = float("nan")


def _i32(x):
    return torch.tensor(np.asarray(x), dtype=torch.int32, device=DEV)


class Case:
    """Caches (optionally paged, pages in random order) whose rows past each length are NaN."""

    def __init__(self, Hq, Hkv, d, bs, lens, paged, seed=0, cap_extra=5, kscale=1.0, scale=None, share=()):
        g = torch.Generator(device=DEV).manual_seed(seed)
        self.g, self.Hq, self.Hkv, self.d, self.bs, self.lens = g, Hq, Hkv, d, bs, list(lens)
        self.B = B = len(lens)
        cap = max(max(lens), 1) + cap_extra
        maxnb = -(-cap // bs)
        self.k = [self.randn(Hkv, n, d) * kscale for n in lens]
        self.v = [self.randn(Hkv, n, d) for n in lens]
        for first, other, tokens in share:  # the first `tokens` tokens of `other` are those of `first`
            self.k[other][:, :tokens], self.v[other][:, :tokens] = self.k[first][:, :tokens], self.v[first][:, :tokens]
        table = None
        if paged:
            held = [-(-n // bs) for n in lens]
            pages = sum(held) + 3
            order = np.random.RandomState(seed).permutation(pages)
            t, at = np.full((B, maxnb), -1, np.int32), 0
            for b in range(B):
                t[b, :held[b]] = order[at:at + held[b]]
                at += held[b]
            table = _i32(t)
            shape = (pages, Hkv, bs, d)
        else:
            pages, shape = 0, (B, Hkv, cap, d)
        self.table = table
        self.kc = torch.full(shape, NAN, dtype=torch.bfloat16, device=DEV)
        self.vc = torch.full(shape, NAN, dtype=torch.bfloat16, device=DEV)
        for b, n in enumerate(lens):
            for j in range(-(-n // bs)):
                a, z = j * bs, min(n, (j + 1) * bs)
                for c, x in ((self.kc, self.k[b]), (self.vc, self.v[b])):
                    if paged:
                        c[int(t[b, j]), :, :z - a] = x[:, a:z]
                    else:
                        c[b, :, a:z] = x[:, a:z]
        self.dims = prr.Dims(B=B, Hq=Hq, Hkv=Hkv, d=d, bs=bs, cap_tokens=cap, K=8, P=0, scale=scale, pages=pages,
                             block_table=None if table is None else table.data_ptr())
        self.scale = 1 / math.sqrt(d) if scale is None else scale
        self.seq_lens = _i32(lens)

    def randn(self, *shape):
        return torch.randn(shape, generator=self.g, device=DEV, dtype=torch.bfloat16)

    def ws(self, rows=1):
        return torch.zeros(prr.prr_serving_workspace_bytes(self.dims, max(rows, 1)), dtype=torch.uint8, device=DEV)

    def exact(self, q, b, n):
        """One query row [Hq][d] over the first n tokens of b: out, lse and their tolerances."""
        G = self.Hq // self.Hkv
        qd = q.double().view(self.Hkv, G, self.d)
        k, v = self.k[b][:, :n].double(), self.v[b][:, :n].double()
        s = torch.einsum("hgd,hnd->hgn", qd, k) * self.scale
        lse = torch.logsumexp(s, -1)
        w = torch.exp(s - lse[..., None])
        out = torch.einsum("hgn,hnd->hgd", w, v)
        tol = 2.0 ** -8 * (torch.einsum("hgn,hnd->hgd", w, v.abs()) + out.abs()) * 1.02 + 1e-6
        big = torch.einsum("hgd,hnd->hgn", qd.abs(), k.abs()).amax(-1) * abs(self.scale)
        ltol = (self.d + 2) * 2.0 ** -24 * big + 2.0 ** -21 * (1 + lse.abs()) + n * 2.0 ** -24
        # an error in a logit is one in its weight too
        tol = tol + (2 * ltol[..., None]) * torch.einsum("hgn,hnd->hgd", w, v.abs())
        f = lambda x: x.reshape(self.Hq, -1)  # noqa: E731
        return f(out), lse.reshape(-1), f(tol), ltol.reshape(-1)

    def check(self, q, out, lse, rows):
        """rows: (row of out, sequence, tokens seen)"""
        for row, b, n in rows:
            o, l, tol, ltol = self.exact(q[row], b, n)
            bad = (out[row].double() - o).abs() - tol
            assert bool((bad <= 0).all()), (row, b, n, float(bad.max()), float(tol.max()))
            if lse is not None:
                off = (lse[row].double() - l).abs() - ltol
                assert bool((off <= 0).all()), (row, b, n, float(off.max()))


def _prompt(c, new, q=None, lse=True, stream=None, tail=3, ws=None):
    """Attend the newest new[b] rows of each sequence; `tail` more rows of q belong to no one."""
    T = sum(new)
    q = c.randn(T + tail, c.Hq, c.d) if q is None else q
    qb = np.concatenate([[0], np.cumsum(new)])
    out = torch.full((q.shape[0], c.Hq, c.d), 7.0, dtype=torch.bfloat16, device=DEV)
    L = torch.full((q.shape[0], c.Hq), 7.0, device=DEV) if lse else None
    ws = c.ws(q.shape[0]) if ws is None else ws
    qb_dev = _i32(qb)
    if stream is not None:  # what the call reads and writes is made on the current stream
        stream.wait_stream(torch.cuda.current_stream())
    prr.prr_attend_prompt(c.dims, q, qb_dev, c.seq_lens, c.kc, c.vc, out, L, ws, stream)
    return q, qb, out, L, ws


def _some(rows, most=48):
    rows = list(rows)
    if len(rows) <= most:
        return rows
    keep = {0, 1, len(rows) - 1} | set(np.random.RandomState(1).choice(len(rows), most, replace=False).tolist())
    return [rows[i] for i in sorted(keep)]


@pytest.mark.parametrize("Hq,Hkv,d,bs,paged,new,old", [
    (1, 1, 64, 64, False, [1], [0]),
    (4, 1, 64, 64, True, [37], [0]),
    (4, 1, 128, 128, True, [1, 128, 129], [0, 0, 0]),
    (32, 8, 128, 64, True, [300, 1, 0, 513, 64], [0, 700, 90, 0, 64]),
    (16, 2, 128, 128, False, [17, 260], [1000, 3]),
    (6, 2, 64, 128, True, [255, 1], [130, 4000]),
    (5, 1, 128, 64, False, [200], [77]),
    (14, 2, 64, 64, True, [101, 9], [0, 511]),
    (2, 2, 128, 64, True, [700], [0]),
    (8, 4, 64, 128, False, [1, 1, 1], [0, 127, 128]),
])
def test_attend_prompt(Hq, Hkv, d, bs, paged, new, old):
    c = Case(Hq, Hkv, d, bs, [a + b for a, b in zip(new, old)], paged)
    q, qb, out, lse, ws = _prompt(c, new)
    c.check(q, out, lse, _some((int(qb[b]) + i, b, old[b] + i + 1) for b in range(c.B) for i in range(new[b])))
    assert bool((out[int(qb[-1]):] == 7).all()) and bool((lse[int(qb[-1]):] == 7).all())  # rows of no sequence
    assert prr.prr_get_device_status(ws) == 0


def test_attend_prompt_of_several_thousand_rows():
    new = [5000, 1, 3333]
    c = Case(8, 2, 128, 64, [5000, 9000, 3400], True, seed=3)
    q, qb, out, lse, ws = _prompt(c, new)
    old = [0, 8999, 67]
    c.check(q, out, lse, _some(((int(qb[b]) + i, b, old[b] + i + 1) for b in range(3) for i in range(new[b])), 80))
    assert prr.prr_get_device_status(ws) == 0


@pytest.mark.parametrize("kscale,scale", [(20.0, None), (1.0, 0.0), (1.0, -0.3), (0.0, None), (300.0, None)])
def test_attend_prompt_extreme_logits(kscale, scale):
    c = Case(8, 2, 128, 64, [700], True, kscale=kscale, scale=scale)
    q, qb, out, lse, _ = _prompt(c, [400])
    c.check(q, out, lse, _some((i, 0, 300 + i + 1) for i in range(400)))


def test_attend_prompt_logits_that_grow_along_the_context():
    """Every block's logits are above all before it: the running maximum moves each time."""
    c = Case(4, 1, 64, 64, [2000], False)
    q = c.randn(500, 4, 64).abs() + 0.5
    ramp = (torch.arange(2000, device=DEV) / 100)[None, :, None]
    c.k[0] = (torch.full_like(c.k[0], 0.25) + ramp * 0.05).bfloat16()
    c.kc[0, :, :2000] = c.k[0]
    q, qb, out, lse, _ = _prompt(c, [500], q=q)
    c.check(q, out, lse, _some((i, 0, 1500 + i + 1) for i in range(500)))


def test_attend_prompt_strided_rows_and_no_lse():
    c = Case(8, 2, 128, 64, [333], True)
    wide = c.randn(333, 12, 128)
    q, qb, out, lse, _ = _prompt(c, [333], q=wide[:, :8], lse=False)
    c.check(q, out, None, _some((i, 0, i + 1) for i in range(333)))


def test_attend_prompt_same_bits_twice_on_a_side_stream_and_in_a_graph():
    c = Case(32, 8, 128, 64, [900, 40], True)
    q, qb, out, lse, ws = _prompt(c, [650, 3])
    torch.cuda.synchronize()
    st = torch.cuda.Stream()
    _, _, out2, lse2, _ = _prompt(c, [650, 3], q=q, stream=st)
    torch.cuda.synchronize()
    assert torch.equal(out[:653], out2[:653]) and torch.equal(lse[:653], lse2[:653])
    out3, lse3, qb3 = torch.zeros_like(out), torch.zeros_like(lse), _i32(qb)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        prr.prr_attend_prompt(c.dims, q, qb3, c.seq_lens, c.kc, c.vc, out3, lse3, ws)
    for _ in range(3):
        out3.zero_()
        graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(out[:653], out3[:653]) and torch.equal(lse[:653], lse3[:653])
    # another batch behind the same graph: its rows are read on the device
    qb3.copy_(_i32([0, 10, 13]))
    graph.replay()
    c.check(q, out3, lse3, [(i, 0, 890 + i + 1) for i in range(10)] + [(10 + i, 1, 37 + i + 1) for i in range(3)])
    assert prr.prr_get_device_status(ws) == 0


@pytest.mark.parametrize("change,code", [
    (dict(qb=[0, 5, 20]), 5), (dict(qb=[0, -1, 3]), 5), (dict(lens=[50, 2]), 1), (dict(lens=[50, 0]), 1),
    (dict(lens=[50, 1 << 20]), 1),
])
def test_attend_prompt_bad_sequence_is_skipped(change, code):
    c = Case(4, 1, 64, 64, [50, 30], True)
    q = c.randn(8, 4, 64)
    out = torch.full((8, 4, 64), 7.0, dtype=torch.bfloat16, device=DEV)
    ws = c.ws(8)
    prr.prr_attend_prompt(c.dims, q, _i32(change.get("qb", [0, 5, 8])), _i32(change.get("lens", [50, 30])), c.kc, c.vc,
                          out, None, ws)
    assert prr.prr_get_device_status(ws) == code
    assert bool((out[5:] == 7).all())
    if change.get("qb", [0, 5])[1] == 5:
        c.check(q, out, None, [(i, 0, 45 + i + 1) for i in range(5)])


def test_attend_prompt_bad_page_sets_status():
    c = Case(4, 1, 64, 64, [200], True)
    c.table[0, 1] = 10 ** 6
    _, _, _, _, ws = _prompt(c, [5])
    assert prr.prr_get_device_status(ws) == 5


def _shared(c, members, gb, sb, q=None, ws=None):
    q = c.randn(c.B, c.Hq, c.d) if q is None else q
    out = torch.full((c.B, c.Hq, c.d), 7.0, dtype=torch.bfloat16, device=DEV)
    lse = torch.full((c.B, c.Hq), 7.0, device=DEV)
    ws = c.ws() if ws is None else ws
    prr.prr_attend_shared(c.dims, q, _i32(members), _i32(gb), _i32(sb), c.seq_lens, c.kc, c.vc, out, lse, ws)
    return q, out, lse, ws


@pytest.mark.parametrize("Hq,Hkv,d,bs,paged,prefix,own", [
    ([4, 1, 64, 64, True, [2], [[0, 1, 63, 64, 65]]]),
    ([32, 8, 128, 64, True, [20, 0], [[5, 600, 0, 129], [1, 77]]]),
    ([16, 2, 128, 128, False, [3, 1, 7], [[1] * 40, [300], [0, 0, 5]]]),
    ([6, 2, 64, 128, True, [9, 2], [[3, 2, 1], [2000]]]),
    ([7, 1, 128, 64, False, [0], [[1, 0, 500, 1300]]]),
    ([8, 8, 64, 64, True, [33], [[4] * 260]]),
    ([4, 1, 64, 64, True, [300], [[0]]]),
    ([12, 4, 128, 64, True, [5, 9, 3], [[], [7, 70], []]]),  # groups of no one
    ([7, 1, 128, 64, True, [19] * 4, [[1, 2, 3, 4] * 3 + [1]] * 4]),  # a CTA whose only piece is one step of few rows
])
def test_attend_shared(Hq, Hkv, d, bs, paged, prefix, own):
    lens, gb, share = [], [0], []
    for pb, tails in zip(prefix, own):
        first = len(lens)
        lens += [pb * bs + t for t in tails]
        share += [(first, b, pb * bs) for b in range(first + 1, len(lens))]
        gb.append(len(lens))
    lens += [50]  # a sequence of no group
    c = Case(Hq, Hkv, d, bs, lens, paged, share=share)
    # the groups' members are not in the batch's order
    members = [b for i in range(len(prefix)) for b in np.random.RandomState(i).permutation(np.arange(gb[i], gb[i + 1]))]
    q, out, lse, ws = _shared(c, members, gb, prefix)
    c.check(q, out, lse, _some((b, b, lens[b]) for b in range(c.B - 1) if lens[b]))
    for b in range(c.B - 1):
        if lens[b] == 0:
            assert bool((out[b] == 0).all()) and bool((lse[b] == -math.inf).all())
    assert bool((out[-1] == 7).all()) and bool((lse[-1] == 7).all())
    assert prr.prr_get_device_status(ws) == 0


def test_a_batch_of_three_thousand_single_tokens():
    """More sequences than the plan keeps on chip, through both attention calls; most CTAs have many pieces."""
    B = 3000
    lens = [int(x) for x in np.random.RandomState(0).randint(1, 200, B)]
    c = Case(4, 2, 64, 64, lens, True)
    q, qb, out, lse, ws = _prompt(c, [1] * B, tail=0)
    rows = _some(((b, b, lens[b]) for b in range(B)), 40)
    c.check(q, out, lse, rows)
    _, out2, lse2, ws2 = _shared(c, np.random.RandomState(1).permutation(B), [0, B], [0], q=q)
    c.check(q, out2, lse2, rows)
    assert (out.float() - out2.float()).abs().max() < 0.05 and bool((lse - lse2).abs().max() < 1e-4)
    assert prr.prr_get_device_status(ws) == 0 and prr.prr_get_device_status(ws2) == 0


def test_attend_shared_reads_the_prefix_through_its_first_member():
    """The other members' copies of a shared prefix are not read: they may hold anything."""
    c = Case(4, 1, 64, 64, [200, 210, 150], False, share=[(0, 1, 128), (0, 2, 128)])
    c.kc[1:, :, :128], c.vc[1:, :, :128] = NAN, NAN
    q, out, lse, ws = _shared(c, [0, 1, 2], [0, 3], [2])
    c.check(q, out, lse, [(b, b, c.lens[b]) for b in range(3)])


def test_attend_shared_equals_itself_in_a_graph_and_with_a_sequence_listed_twice():
    c = Case(32, 8, 128, 64, [1100, 1200, 1030], True, share=[(0, 1, 1024), (0, 2, 1024)])
    q, out, lse, ws = _shared(c, [0, 1, 2], [0, 3], [16])
    out2, lse2 = torch.zeros_like(out), torch.zeros_like(lse)
    m, gb, sb = _i32([0, 1, 2]), _i32([0, 3]), _i32([16])
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        prr.prr_attend_shared(c.dims, q, m, gb, sb, c.seq_lens, c.kc, c.vc, out2, lse2, ws)
    graph.replay()
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, out2) and torch.equal(lse, lse2)
    _, out3, lse3, _ = _shared(c, [1, 1, 0], [0, 3], [16], q=q)
    c.check(q, out3, lse3, [(0, 0, 1100), (1, 1, 1200)])
    assert bool((out3[2] == 7).all())


@pytest.mark.parametrize("members,gb,sb,lens,code,good", [
    ([0, 9, 2], [0, 3], [1], None, 5, [0, 2]), ([-1, 1, 2], [0, 3], [1], None, 5, []),
    ([0, 1, 2], [0, 3], [3], None, 5, [0, 1]), ([0, 1, 2], [0, 3], [-1], None, 5, []),
    ([0, 1, 2], [0, 4], [1], None, 5, []), ([0, 1, 2], [0, 1, 3], [1, 9], None, 5, [0]),
    ([-1, 1, 2], [0, 3], [0], None, 5, [1, 2]),  # nothing is read through the first member
    ([0, 1, 2], [0, 3], [1], [200, -1, 130], 1, [0, 2]), ([0, 1, 2], [0, 3], [1], [200, 1 << 29, 130], 1, [0, 2]),
])
def test_attend_shared_bad_entries_are_skipped(members, gb, sb, lens, code, good):
    c = Case(4, 1, 64, 64, [200, 210, 130], False, share=[(0, 1, 128), (0, 2, 128)])
    if lens:
        c.seq_lens = _i32(lens)
    q, out, lse, ws = _shared(c, members, gb, sb)
    assert prr.prr_get_device_status(ws) == code
    if sb == [3]:  # three blocks of the group are read through its first member, though only two are alike
        c.k[1][:, :192], c.v[1][:, :192] = c.k[0][:, :192], c.v[0][:, :192]
    c.check(q, out, lse, [(b, b, c.lens[b]) for b in good])
    for b in set(range(3)) - set(good):
        assert bool((out[b] == 7).all()) and bool((lse[b] == 7).all()), b


# ----------------------------------------------------------------------------- appending prompts

@pytest.mark.parametrize("Hkv,d,bs,paged,new,old", [
    (1, 64, 64, False, [1], [0]), (2, 128, 64, True, [100, 0, 1, 300], [30, 5, 63, 64]),
    (8, 128, 128, True, [129, 1000], [0, 127]), (3, 64, 128, False, [7, 250], [500, 0]),
])
@pytest.mark.parametrize("strided", [False, True])
def test_append_prompt(Hkv, d, bs, paged, new, old, strided):
    ends = [a + b for a, b in zip(new, old)]
    c = Case(2 * Hkv, Hkv, d, bs, ends, paged)
    T = sum(new)
    qb = np.concatenate([[0], np.cumsum(new)])
    wide = c.randn(T + 2, 4 * Hkv, d)
    k, v = wide[:, 2 * Hkv:3 * Hkv], wide[:, 3 * Hkv:]
    if not strided:
        k, v = k.contiguous(), v.contiguous()
    maxnb = c.dims.maxnb
    summ = torch.full((c.B, Hkv, maxnb, 2, d), 99.0, dtype=torch.bfloat16, device=DEV)
    kc, vc, want = c.kc.clone(), c.vc.clone(), summ.clone()
    for b in range(c.B):
        c.k[b][:, old[b]:] = k[int(qb[b]):int(qb[b + 1])].transpose(0, 1)
        c.v[b][:, old[b]:] = v[int(qb[b]):int(qb[b + 1])].transpose(0, 1)
        for j in range(-(-ends[b] // bs)):
            a, z = j * bs, min(ends[b], (j + 1) * bs)
            page = int(c.table[b, j]) if paged else b
            lo = 0 if paged else a
            kc[page, :, lo:lo + z - a], vc[page, :, lo:lo + z - a] = c.k[b][:, a:z], c.v[b][:, a:z]
            if min(old[b], z) > a:  # what was cached is summarised already
                have = c.k[b][:, a:min(old[b], z)]
                summ[b, :, j, 0], summ[b, :, j, 1] = have.amin(1), have.amax(1)
            want[b, :, j, 0], want[b, :, j, 1] = c.k[b][:, a:z].amin(1), c.k[b][:, a:z].amax(1)
    lens, ws = _i32(old), c.ws(T + 2)
    prr.prr_append_prompt(c.dims, k, v, _i32(qb), lens, c.kc, c.vc, summ, ws)
    assert lens.tolist() == ends
    same = lambda a, b: bool(((a == b) | (a.isnan() & b.isnan())).all())  # noqa: E731
    assert same(c.kc, kc) and same(c.vc, vc)
    assert torch.equal(summ, want)
    assert prr.prr_get_device_status(ws) == 0


@pytest.mark.parametrize("lens,qb,code,after", [
    ([50, 62], [0, 4, 8], 1, [54, 62]), ([-1, 0], [0, 4, 8], 1, [-1, 4]), ([0, 0], [0, 4, 9], 5, [4, 0]),
    ([10, 0], [0, 4, 8], 5, [14, 4]),
])
def test_append_prompt_refuses_what_does_not_fit(lens, qb, code, after):
    """A full sequence, a negative length, rows past the array, a block without a page."""
    dims = prr.Dims(B=2, Hq=2, Hkv=1, d=64, bs=64, cap_tokens=64, K=1, P=0, pages=2)
    table = _i32([[1], [0 if lens[0] != 10 else -1]])
    import dataclasses
    dims = dataclasses.replace(dims, block_table=table.data_ptr())
    kc = torch.zeros(2, 1, 64, 64, dtype=torch.bfloat16, device=DEV)
    vc, k = torch.zeros_like(kc), torch.ones(8, 1, 64, dtype=torch.bfloat16, device=DEV)
    L = _i32(lens)
    ws = torch.zeros(prr.prr_serving_workspace_bytes(dims, 8), dtype=torch.uint8, device=DEV)
    prr.prr_append_prompt(dims, k, k, _i32(qb), L, kc, vc, None, ws)
    assert prr.prr_get_device_status(ws) == code
    assert L.tolist() == after
    assert int(kc.sum()) == 64 * (8 if False else sum(max(a - b, 0) for a, b, p in zip(after, lens, table.tolist()) if p[0] >= 0))


# ----------------------------------------------------------------------------- pages

class Model:
    """The page calls restated one entry at a time, on the host."""

    def __init__(self, B, maxnb, pages, bs):
        self.B, self.maxnb, self.pages, self.bs = B, maxnb, pages, bs
        self.table = -np.ones((B, maxnb), np.int64)
        self.refs = np.zeros(pages, np.int64)
        self.lens = np.zeros(B, np.int64)
        self.content = {}  # page -> what it holds

    def free(self):
        return [i for i in range(self.pages) if self.refs[i] == 0]

    def reserve(self, want):
        holes = [(b, j) for b in range(self.B) for j in range(-(-int(self.lens[b]) // self.bs), -(-int(want[b]) // self.bs))
                 if want[b] > 0 and self.table[b, j] < 0]
        free = self.free()
        if len(free) < len(holes):
            return False
        for (b, j), pg in zip(holes, free):
            self.table[b, j], self.refs[pg] = pg, 1
        return True

    def fork(self, parents, children):
        n = [int(self.lens[p]) for p in parents]
        free = self.free()
        tails = [i for i in range(len(n)) if n[i] % self.bs]
        if len(free) < len(tails):
            return False
        give = dict(zip(tails, free))
        for i, (p, c) in enumerate(zip(parents, children)):
            full = n[i] // self.bs
            for j in range(full):
                self.table[c, j] = self.table[p, j]
                self.refs[self.table[p, j]] += 1
            if i in give:
                self.content[give[i]] = self.content[int(self.table[p, full])]
                self.table[c, full], self.refs[give[i]] = give[i], 1
            self.lens[c] = n[i]
        return True

    def release(self, seqs):
        for b in set(seqs):
            for pg in self.table[b][self.table[b] >= 0]:
                self.refs[pg] -= 1
            self.table[b], self.lens[b] = -1, 0

    def compact(self):
        live = [i for i in range(self.pages) if self.refs[i] > 0]
        L = len(live)
        to = dict(zip([i for i in live if i >= L], [i for i in self.free() if i < L]))
        remap = np.array([to.get(i, i if self.refs[i] > 0 else -1) for i in range(self.pages)])
        for s, t in to.items():
            self.refs[t], self.refs[s] = self.refs[s], 0
            self.content.pop(t, None)
            if s in self.content:
                self.content[t] = self.content[s]
        self.table = np.where(self.table >= 0, remap[self.table], -1)
        return remap, L


@pytest.mark.parametrize("seed,B,pages,d,bs", [(0, 6, 40, 64, 64), (1, 12, 2500, 64, 128), (2, 3, 9, 128, 64),
                                               (3, 40, 1030, 64, 64)])
def test_pages_over_a_random_life(seed, B, pages, d, bs):
    r = np.random.RandomState(seed)
    maxnb, Hkv, P = max(4, pages // 5), 2, 4
    table, refs, lens = _i32(-np.ones((B, maxnb))), _i32(np.zeros(pages)), _i32(np.zeros(B))
    dims = prr.Dims(B=B, Hq=4, Hkv=Hkv, d=d, bs=bs, cap_tokens=maxnb * bs, K=2, P=P, pages=pages,
                    block_table=table.data_ptr())
    kc = torch.zeros(pages, Hkv, bs, d, dtype=torch.bfloat16, device=DEV)
    vc = torch.zeros_like(kc)
    summ = torch.zeros(B, Hkv, maxnb, 2, d, dtype=torch.bfloat16, device=DEV)
    ema = torch.zeros(B, Hkv, maxnb, dtype=torch.float64, device=DEV)
    pred = torch.zeros(B, Hkv, P, dtype=torch.int32, device=DEV)
    bufs = prr.cache_buffers(kc, vc, table, refs, lens, summ, ema, pred)
    ws = torch.zeros(prr.prr_serving_workspace_bytes(dims, 1), dtype=torch.uint8, device=DEV)
    m, mark = Model(B, maxnb, pages, bs), 0
    for step in range(60):
        what = r.choice(["grow", "grow", "fork", "release", "compact"])
        full = False
        if what == "grow":
            want = np.where(r.rand(B) < 0.5, m.lens + r.randint(0, 3 * bs, B), 0).clip(0, maxnb * bs)
            full = not m.reserve(want)
            prr.prr_cache_reserve(dims, _i32(want), bufs, ws)
            if not full:  # every sequence that asked grows into its pages; its new last block gets a mark
                m.lens = np.maximum(m.lens, want)
                lens.copy_(_i32(m.lens))
                for b in range(B):
                    if want[b] > 0 and m.lens[b] > 0:
                        mark = mark % 250 + 1
                        pg = int(m.table[b, (m.lens[b] - 1) // bs])
                        m.content[pg] = mark
                        kc[pg], vc[pg] = mark, -mark
        elif what == "fork":
            empty, used = np.nonzero(m.lens == 0)[0], np.nonzero(m.lens > 0)[0]
            empty = [b for b in empty if m.table[b, 0] < 0]
            if not len(empty) or not len(used):
                continue
            kids = list(r.permutation(empty)[:r.randint(1, len(empty) + 1)])
            pars = [int(r.choice(used)) for _ in kids]
            summ.copy_(torch.randint(-9, 9, summ.shape, device=DEV))
            ema.uniform_()
            pred.random_(0, 99)
            s0, e0, p0 = summ.clone(), ema.clone(), pred.clone()
            full = not m.fork(pars, kids)
            prr.prr_cache_fork(dims, _i32(pars), _i32(kids), bufs, ws)
            if not full:
                for p, k in zip(pars, kids):
                    nb = -(-int(m.lens[p]) // bs)
                    s0[k, :, :nb], e0[k, :, :nb], e0[k, :, nb:], p0[k] = s0[p, :, :nb], e0[p, :, :nb], 0, p0[p]
            assert torch.equal(summ, s0) and torch.equal(ema, e0) and torch.equal(pred, p0)
        elif what == "release":
            seqs = list(r.permutation(B)[:r.randint(1, max(2, B // 2))])
            m.release(seqs)
            prr.prr_cache_release(dims, _i32((seqs + seqs[:1])[:B]), bufs, ws)
            assert not ema[seqs].any() and bool((pred[seqs] == _i32(np.arange(P))).all())
        else:
            remap, n = torch.zeros(pages, dtype=torch.int32, device=DEV), _i32([0])
            want, L = m.compact()
            prr.prr_cache_compact(dims, bufs, remap, n, ws)
            assert int(n) == L and np.array_equal(remap.cpu().numpy(), want)
        assert prr.prr_get_device_status(ws) == (6 if full else 0), (step, what)
        if full:
            prr.prr_workspace_init(ws)
        assert np.array_equal(table.cpu().numpy(), m.table), (step, what)
        assert np.array_equal(refs.cpu().numpy(), m.refs), (step, what)
        assert np.array_equal(lens.cpu().numpy(), m.lens), (step, what)
        for pg in {int(x) for x in m.table[m.table >= 0].reshape(-1)} & set(m.content):
            assert bool((kc[pg] == m.content[pg]).all()) and bool((vc[pg] == -m.content[pg]).all()), (step, what, pg)


def test_fork_refuses_bad_entries_and_does_the_others():
    table, refs, lens = _i32([[0, 1], [-1, -1], [-1, -1], [2, -1], [-1, -1]]), _i32([1, 1, 1, 0, 0, 0]), _i32([70, 0, 0, 5, 0])
    dims = prr.Dims(B=5, Hq=1, Hkv=1, d=64, bs=64, cap_tokens=128, K=1, P=0, pages=6, block_table=table.data_ptr())
    kc = torch.arange(6, device=DEV).view(6, 1, 1, 1).expand(6, 1, 64, 64).bfloat16().contiguous()
    vc = kc.clone()
    bufs = prr.cache_buffers(kc, vc, table, refs, lens)
    ws = torch.zeros(prr.prr_serving_workspace_bytes(dims, 1), dtype=torch.uint8, device=DEV)
    # child not empty; the same child twice; parent out of range; a child of the call as parent
    prr.prr_cache_fork(dims, _i32([0, 0, 3, 7, 1]), _i32([3, 1, 1, 2, 4]), bufs, ws)
    assert prr.prr_get_device_status(ws) == 5
    assert table.tolist() == [[0, 1], [0, 3], [-1, -1], [2, -1], [-1, -1]]
    assert refs.tolist() == [2, 1, 1, 1, 0, 0] and lens.tolist() == [70, 70, 0, 5, 0]
    assert bool((kc[3] == 1).all()) and bool((vc[3] == 1).all())


def test_release_reports_a_count_that_did_not_know_of_a_row():
    table, refs, lens = _i32([[0, 5], [1, -1]]), _i32([0, 1]), _i32([70, 5])
    dims = prr.Dims(B=2, Hq=1, Hkv=1, d=64, bs=64, cap_tokens=128, K=1, P=0, pages=2, block_table=table.data_ptr())
    bufs = prr.cache_buffers(block_table=table, page_refs=refs, seq_lens=lens)
    ws = torch.zeros(prr.prr_serving_workspace_bytes(dims, 1), dtype=torch.uint8, device=DEV)
    prr.prr_cache_release(dims, _i32([0, 1]), bufs, ws)
    assert prr.prr_get_device_status(ws) == 5
    assert refs.tolist() == [0, 0] and lens.tolist() == [0, 0] and bool((table == -1).all())


@pytest.mark.parametrize("selector,n_rep", [("per_head", 0), ("representative", 3)])
def test_fork_and_release_carry_the_state_of_every_selector(selector, n_rep):
    B, Hq, Hkv, d, bs, maxnb, P, pages = 3, 4, 2, 64, 64, 4, 5, 12
    S = Hq if selector == "per_head" else Hkv
    table, refs, lens = _i32([[3, 7, 1, -1], [-1] * 4, [-1] * 4]), _i32(np.zeros(pages)), _i32([150, 0, 0])
    refs[[3, 7, 1]] = 1
    rep = torch.randint(0, bs, (B, Hkv, maxnb, max(n_rep, 1)), dtype=torch.uint8, device=DEV)
    dims = prr.Dims(B=B, Hq=Hq, Hkv=Hkv, d=d, bs=bs, cap_tokens=maxnb * bs, K=2, P=P, pages=pages, selector=selector,
                    n_rep=n_rep, block_table=table.data_ptr(), rep_offsets=rep.data_ptr() if n_rep else None)
    kc = torch.randn(pages, Hkv, bs, d, device=DEV).bfloat16()
    vc = torch.randn(pages, Hkv, bs, d, device=DEV).bfloat16()
    ema = torch.rand(B, S, maxnb, dtype=torch.float64, device=DEV)
    pred = torch.randint(0, 9, (B, S, P), dtype=torch.int32, device=DEV)
    rep0, ema0, pred0 = rep.clone(), ema.clone(), pred.clone()
    bufs = prr.cache_buffers(kc, vc, table, refs, lens, None, ema, pred, rep if n_rep else None)
    ws = torch.zeros(prr.prr_serving_workspace_bytes(dims, 1), dtype=torch.uint8, device=DEV)
    prr.prr_cache_fork(dims, _i32([0]), _i32([2]), bufs, ws)
    assert prr.prr_get_device_status(ws) == 0
    assert table.tolist()[2] == [3, 7, 0, -1] and lens.tolist() == [150, 0, 150]
    assert torch.equal(kc[0], kc[1]) and torch.equal(vc[0], vc[1])
    assert torch.equal(ema[2, :, :3], ema0[0, :, :3]) and not ema[2, :, 3].any() and torch.equal(pred[2], pred0[0])
    if n_rep:
        assert torch.equal(rep[2, :, :3], rep0[0, :, :3]) and torch.equal(rep[2, :, 3], rep0[2, :, 3])
    prr.prr_cache_release(dims, _i32([2]), bufs, ws)
    assert refs.tolist()[:8] == [0, 1, 0, 1, 0, 0, 0, 1] and not ema[2].any()
    assert bool((pred[2] == _i32(np.arange(P))).all())
    assert torch.equal(ema[:2], ema0[:2]) and torch.equal(pred[:2], pred0[:2])


def test_caches_past_two_to_the_31_elements():
    """Offsets into K and V of more than 2^31 elements: appended, attended and compacted at the far end."""
    Hkv, d, bs, n = 8, 128, 128, 300
    pages = (1 << 31) // (Hkv * bs * d) + 6
    kc = torch.zeros(pages, Hkv, bs, d, dtype=torch.bfloat16, device=DEV)
    vc = torch.zeros_like(kc)
    used = [pages - 1, pages - 3, pages - 2]
    table, refs = _i32([used]), _i32(np.zeros(pages))
    refs[used] = 1
    dims = prr.Dims(B=1, Hq=8, Hkv=Hkv, d=d, bs=bs, cap_tokens=3 * bs, K=1, P=0, pages=pages, block_table=table.data_ptr())
    lens = _i32([0])
    ws = torch.zeros(prr.prr_serving_workspace_bytes(dims, n), dtype=torch.uint8, device=DEV)
    c = Case(8, Hkv, d, bs, [n], False)
    qb = _i32([0, n])
    prr.prr_append_prompt(dims, c.k[0].transpose(0, 1).contiguous(), c.v[0].transpose(0, 1).contiguous(), qb, lens, kc, vc,
                          None, ws)
    q = c.randn(n, 8, d)
    for _ in range(2):
        out, lse = torch.zeros_like(q), torch.zeros(n, 8, device=DEV)
        prr.prr_attend_prompt(dims, q, qb, lens, kc, vc, out, lse, ws)
        c.check(q, out, lse, _some((i, 0, i + 1) for i in range(n)))
        remap, live = torch.zeros(pages, dtype=torch.int32, device=DEV), _i32([0])
        prr.prr_cache_compact(dims, prr.cache_buffers(kc, vc, table, refs, lens), remap, live, ws)
        assert int(live) == 3 and table.tolist() == [[2, 0, 1]] and refs.tolist()[:4] == [1, 1, 1, 0]
    assert prr.prr_get_device_status(ws) == 0


def test_serving_calls_captured_and_replayed():
    """One graph of a turn -- rows appended and attended, a fork, the shared attention, a release -- replayed twice."""
    B, Hq, Hkv, d, bs, n = 3, 8, 2, 64, 64, 200
    dims = prr.Dims(B=B, Hq=Hq, Hkv=Hkv, d=d, bs=bs, cap_tokens=512, K=2, P=0, pages=20)
    dec = prr.PRRDecoder(dims, empty=True)
    dec.reserve([n, 0, 0])
    c = Case(Hq, Hkv, d, bs, [n], False)
    k, v, q = (x.transpose(0, 1).contiguous() for x in (c.k[0], c.v[0], c.randn(Hq, n, d)))
    qb, kids, pars, mem, gb, sb = _i32([0, n, n, n]), _i32([1, 2]), _i32([0, 0]), _i32([2, 0, 1]), _i32([0, 3]), _i32([3])
    q1 = c.randn(B, Hq, d)
    ws = torch.zeros(prr.prr_serving_workspace_bytes(dec.dims, n), dtype=torch.uint8, device=DEV)
    out, lse, out1, lse1 = (torch.zeros(s, dtype=t, device=DEV) for s, t in (
        ((n, Hq, d), torch.bfloat16), ((n, Hq), torch.float32), ((B, Hq, d), torch.bfloat16), ((B, Hq), torch.float32)))
    lens0, bufs = torch.zeros_like(dec.seq_lens), dec.cache_buffers()

    def turn():
        dec.seq_lens.copy_(lens0)
        prr.prr_append_prompt(dec.dims, k, v, qb, dec.seq_lens, dec.k_cache, dec.v_cache, dec.summ, ws)
        prr.prr_attend_prompt(dec.dims, q, qb, dec.seq_lens, dec.k_cache, dec.v_cache, out, lse, ws)
        prr.prr_cache_fork(dec.dims, pars, kids, bufs, ws)
        prr.prr_attend_shared(dec.dims, q1, mem, gb, sb, dec.seq_lens, dec.k_cache, dec.v_cache, out1, lse1, ws)
        prr.prr_cache_release(dec.dims, kids, bufs, ws)

    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        turn()
    for _ in range(2):
        for t in (out, lse, out1, lse1):
            t.fill_(7)
        graph.replay()
        torch.cuda.synchronize()
        c.check(q, out, lse, _some((i, 0, i + 1) for i in range(n)))
        for b in range(B):
            o, l, tol, ltol = c.exact(q1[b], 0, n)
            assert bool(((out1[b].double() - o).abs() <= tol).all()) and bool(((lse1[b].double() - l).abs() <= ltol).all())
        assert dec.seq_lens.tolist() == [n, 0, 0] and int((dec.page_refs > 0).sum()) == 4
    assert prr.prr_get_device_status(ws) == 0


# ----------------------------------------------------------------------------- together

def test_prompts_forks_shared_attention_and_steps_together():
    """A prompt is appended and attended in two pieces, forked, its children attend the
    shared prefix and take decode steps; a decoder that was given every sequence's tokens
    separately agrees bit for bit on the steps, before and after a compaction."""
    torch.manual_seed(0)
    B, Hq, Hkv, d, bs, n = 4, 8, 2, 64, 64, 700
    cap = 1024
    dims = prr.Dims(B=B, Hq=Hq, Hkv=Hkv, d=d, bs=bs, cap_tokens=cap, K=4, P=4, pages=64)
    dec = prr.PRRDecoder(dims, empty=True)
    qkv = torch.randn(n, Hq + 2 * Hkv, d, device=DEV).bfloat16()
    q, k, v = qkv[:, :Hq], qkv[:, Hq:Hq + Hkv], qkv[:, Hq + Hkv:]
    dec.release(range(1, B))                       # empty already: nothing to give back
    dec.reserve([0, n, 0, 0])
    outs = []
    for a, z in ((0, 450), (450, n)):
        qb = [0, 0, z - a, z - a, z - a]
        dec.append_prompt(k[a:z], v[a:z], qb)
        outs.append(dec.attend_prompt(q[a:z], qb))
    assert dec.seq_lens.tolist() == [0, n, 0, 0]
    c = Case(Hq, Hkv, d, bs, [n], False)
    c.k, c.v = [k.transpose(0, 1)], [v.transpose(0, 1)]
    out, lse = torch.cat([o for o, _ in outs]), torch.cat([x for _, x in outs])
    c.check(q, out, lse, _some((i, 0, i + 1) for i in range(n)))

    dec.fork([1, 1, 1], [0, 2, 3])
    dec.reserve([n + 8] * B)
    flat = prr.PRRDecoder(prr.Dims(B=B, Hq=Hq, Hkv=Hkv, d=d, bs=bs, cap_tokens=cap, K=4, P=4))
    kk = k.transpose(0, 1).expand(B, Hkv, n, d).contiguous()
    flat.prefill(kk, v.transpose(0, 1).expand(B, Hkv, n, d).contiguous(), n)
    dec.seq_lens.tolist()
    flat.pred_buf[0].copy_(dec.pred)
    ks, vs = [k] * B, [v] * B
    for step in range(6):
        qs = torch.randn(B, Hq, d, device=DEV).bfloat16()
        kn, vn = torch.randn(2, B, Hkv, d, device=DEV).bfloat16()
        for x in (dec, flat):
            x.step_fused(qs, k_new=kn, v_new=vn)
        torch.cuda.synchronize()
        assert torch.equal(dec.sel, flat.sel) and torch.equal(dec.pred, flat.pred), step
        assert (dec.out - flat.out).abs().max() < 1e-5, step  # the merge order of partials may differ
        ks = [torch.cat([ks[b], kn[b:b + 1]]) for b in range(B)]
        vs = [torch.cat([vs[b], vn[b:b + 1]]) for b in range(B)]
        if step == 2:
            dec.release([3])
            dec.fork([2], [3])                     # a sample is dropped, another one continued twice
            dec.reserve([n + 8] * B)
            flat.k_cache[3], flat.v_cache[3], flat.summ[3], flat.ema[3] = (
                x[2].clone() for x in (flat.k_cache, flat.v_cache, flat.summ, flat.ema))
            flat.pred[3] = flat.pred[2].clone()
            ks[3], vs[3] = ks[2], vs[2]
            _, live = dec.compact()
            assert int(live) == int((dec.page_refs > 0).sum())
            assert bool((dec.page_refs[:int(live)] > 0).all())
        shared = n // bs
        o, l = dec.attend_shared(qs, [2, 0, 1, 3], [0, 4], [shared])
        c.k, c.v = [x.transpose(0, 1) for x in ks], [x.transpose(0, 1) for x in vs]
        c.check(qs, o, l, [(b, b, n + step + 1) for b in range(B)])
    assert dec.device_status() == 0 and flat.device_status() == 0
    ck = dec.checkpoint()
    other = prr.PRRDecoder(dims, empty=True)
    other.restore(ck)
    assert torch.equal(other.page_refs, dec.page_refs)
    o2, l2 = other.attend_shared(qs, [2, 0, 1, 3], [0, 4], [shared])
    assert torch.equal(o, o2) and torch.equal(l, l2)
