"""GPU tests of the attention over the paged FP8 cache: against the formula in
64 bits, key by key through the block table."""
import math

import pytest
import torch

pytestmark = pytest.mark.gpu
BF16, F8, F32, F64, I32, I64, U8 = (torch.bfloat16, torch.float8_e4m3fn, torch.float32, torch.float64,
                                    torch.int32, torch.int64, torch.uint8)
INF = float("inf")


@pytest.fixture(scope="module")
def jet(torch_cuda):
    import fp8_block_quantized_gb300 as j
    j.load()
    return j


class Batch:
    """Requests of (new tokens, length) each over a randomly ordered cache."""

    def __init__(self, requests, Hq, Hk, D, bs, seed=0, groups=(), behind=0, qpad=0, spare=3, q_std=1.5):
        g = torch.Generator().manual_seed(seed)
        self.Hq, self.Hk, self.D, self.bs = Hq, Hk, D, bs
        new = [n for n, _ in requests]
        self.B, self.T = len(requests), sum(new) + behind
        width = max([1] + [(l + bs - 1) // bs for _, l in requests])
        blocks = sum((l + bs - 1) // bs for _, l in requests) + spare
        ids = torch.randperm(blocks, generator=g).tolist()
        table = torch.full((self.B, width), -1, dtype=I32)
        for b, (_, l) in enumerate(requests):
            for i in range((l + bs - 1) // bs):
                table[b, i] = ids.pop()
        self.S = blocks * bs
        codes = lambda: (torch.randn((self.S, Hk, D), generator=g) * 90).clamp(-448, 448).to(F8).view(U8)
        self.k, self.v = codes().cuda(), codes().cuda()
        self.ks = (torch.rand((Hk,), generator=g) * 0.01 + 0.005).cuda()
        self.vs = (torch.rand((Hk,), generator=g) * 0.01 + 0.005).cuda()
        rows = (torch.randn((self.T, Hq * D + qpad), generator=g) * q_std).to(BF16).cuda()
        self.q = rows[:, :Hq * D].unflatten(1, (Hq, D))
        self.table = table.cuda()
        self.offsets = torch.tensor([0] + new).cumsum(0).cuda()
        self.lengths = torch.tensor([l for _, l in requests], dtype=I32).cuda()
        self.po = self.pl = None
        if groups:                       # (first, end, prefix) each, consecutive
            self.po = torch.tensor([groups[0][0]] + [e for _, e, _ in groups]).cuda()
            self.pl = torch.tensor([p for _, _, p in groups], dtype=I32).cuda()

    def reference(self, scale=None):
        """(out, lse, bound of out, bound of lse) in 64 bits; rows of no request are 0, -inf."""
        Hq, Hk, D, bs = self.Hq, self.Hk, self.D, self.bs
        scale = D ** -0.5 if scale is None else scale
        out = torch.zeros((self.T, Hq, D), dtype=F64)
        lse = torch.full((self.T, Hq), -INF, dtype=F64)
        eo, el = torch.zeros_like(out), torch.zeros_like(lse)
        kd, vd = (c.cpu().view(F8).double() * s.cpu().double()[:, None]
                  for c, s in ((self.k, self.ks), (self.v, self.vs)))
        table, off, length = self.table.cpu().tolist(), self.offsets.tolist(), self.lengths.tolist()
        width = len(table[0])
        po = self.po.tolist() if self.po is not None else []
        pl = self.pl.tolist() if self.po is not None else []
        q = self.q.cpu().double()
        for b in range(self.B):
            prefix, first = 0, b
            for i in range(len(pl)):
                if po[i] <= b < po[i + 1]:
                    first = po[i]
                    prefix = min(max(pl[i], 0), max(0, min(length[first], width * bs)))
            slots, at = [], []
            for p in range(min(length[b], width * bs)):
                e = table[first if p < prefix else b][p // bs]
                if e >= 0 and e * bs + p % bs < self.S:
                    slots.append(e * bs + p % bs)
                    at.append(p)
            at = torch.tensor(at, dtype=I64)
            n = off[b + 1] - off[b]
            for j in range(n):
                see = at <= length[b] - n + j
                if not bool(see.any()):
                    continue
                idx = torch.tensor(slots)[see]
                kk, vv = (t[idx].repeat_interleave(Hq // Hk, 1) for t in (kd, vd))   # [L, Hq, D]
                x = torch.einsum("hd,lhd->hl", q[off[b] + j], kk) * scale
                mag = torch.einsum("hd,lhd->hl", q[off[b] + j].abs(), kk.abs()).amax(1) * scale
                w = torch.softmax(x, 1)
                t = off[b] + j
                out[t] = torch.einsum("hl,lhd->hd", w, vv)
                lse[t] = torch.logsumexp(x, 1)
                # scores: D products summed in binary32, the factor's three roundings; weights: that,
                # e^x to 2^-22, FP16 (2^-11, and 2^-25 of the largest near its smallest), sums of L terms
                L = idx.numel()
                dx = (D + 8) * 2.0 ** -24 * mag + 2.0 ** -22 * x.abs().amax(1)
                rel = 2.0 ** -11 + 2 * dx + 2.0 ** -21 + 2 * L * 2.0 ** -24
                some = torch.einsum("hl,lhd->hd", w, vv.abs())
                eo[t] = 2.0 ** -8 * out[t].abs() + rel[:, None] * some + 2.0 ** -25 * vv.abs().sum(0) * w.amax(1)[:, None]
                el[t] = dx + 2.0 ** -21 + L * 2.0 ** -24 + 2.0 ** -22 * lse[t].abs()
        return out, lse, eo, el

    def call(self, jet, **kw):
        out = torch.full((self.T, self.Hq, self.D), 7.0, dtype=BF16, device="cuda")
        lse = torch.full((self.T, self.Hq), 7.0, device="cuda")
        jet.jet_kv_attention(self.q, self.k, self.v, self.ks, self.vs, self.table, self.bs, self.offsets,
                             self.lengths, out, lse, self.po, self.pl, **kw)
        torch.cuda.synchronize()
        return out, lse

    def check(self, jet, **kw):
        out, lse = self.call(jet, **kw)
        ro, rl, eo, el = self.reference(kw.get("scale"))
        end = int(self.offsets[-1])
        got, gl = out.cpu().double(), lse.cpu().double()
        assert (got[end:] == 7).all() and (gl[end:] == 7).all()      # rows of no request
        got, gl, ro, rl, eo, el = (t[:end] for t in (got, gl, ro, rl, eo, el))
        assert torch.equal(rl == -INF, gl == -INF)
        some = rl > -INF
        assert (got[~some] == 0).all()
        assert ((got - ro).abs() <= eo)[some].all(), ((got - ro).abs() - eo).max()
        assert ((gl - rl).abs() <= el)[some].all(), ((gl - rl).abs() - el)[some].max()
        return out, lse


DECODE = [(1, 1), (1, 2), (1, 31), (1, 32), (1, 33), (1, 127), (1, 128), (1, 129), (1, 300), (1, 64)]


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("Hq,Hk", [(1, 1), (4, 4), (6, 2), (8, 1), (24, 1), (32, 8)])
def test_decode(jet, D, Hq, Hk):
    Batch(DECODE, Hq, Hk, D, 16, seed=D + Hq).check(jet)


@pytest.mark.parametrize("bs", [1, 8, 24, 64, 1000])
def test_block_sizes(jet, bs):
    Batch([(1, 200), (3, 77), (1, 1), (2, 130)], 8, 2, 128, bs, seed=bs).check(jet)


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("Hq,Hk", [(2, 2), (6, 2), (8, 1)])
def test_chunks(jet, D, Hq, Hk):
    """Any number of new tokens, with and without keys before them."""
    Batch([(5, 5), (17, 40), (0, 50), (1, 1), (40, 200), (130, 131), (2, 400)], Hq, Hk, D, 16,
          seed=3 * D + Hq).check(jet)


@pytest.mark.parametrize("requests", [[(1, 1)], [(1, 4096)], [(300, 300)], [(16, 16)] * 3, [(0, 9)],
                                      [(1, 700)] * 40, [(3, 64), (0, 0), (0, 0), (1, 65)]])
def test_batches(jet, requests):
    Batch(requests, 8, 2, 128, 16, seed=len(requests)).check(jet)


def test_rows_behind_the_last_request_and_strided_queries(jet):
    Batch([(1, 40), (2, 50)], 8, 2, 128, 16, seed=1, behind=5, qpad=64).check(jet)


def test_queries_that_see_no_key(jet):
    """Lengths of zero, below the number of new tokens, and tables without blocks."""
    b = Batch([(1, 20), (3, 3), (2, 40), (1, 5), (4, 30)], 4, 2, 64, 8, seed=2)
    b.lengths[0], b.lengths[1] = 0, 1
    b.lengths[3] = -4
    b.table[4] = -1
    out, lse = b.check(jet)
    assert (lse[0] == -INF).all() and (lse[1:3] == -INF).all() and (lse[3] > -INF).all()


def test_keys_without_a_slot_are_left_out(jet):
    b = Batch([(1, 200), (4, 90), (1, 300)], 8, 4, 128, 16, seed=5)
    b.table[0, 2] = -1                     # a missing block
    b.table[1, 0] = -7
    b.table[2, 5] = b.S // b.bs            # a block past the cache
    b.table[2, 6] = 2 ** 31 - 1
    b.lengths[0] = 10000                   # past the table's width
    b.check(jet)


def test_nan_behind_the_length_does_not_show(jet):
    """What lies in unused slots of the last block, and in blocks nobody holds."""
    b = Batch([(1, 37), (2, 130)], 4, 2, 128, 64, seed=6)
    want = b.call(jet)
    used = torch.zeros((b.S,), dtype=torch.bool)
    for r, l in enumerate(b.lengths.tolist()):
        for p in range(l):
            used[int(b.table[r, p // b.bs]) * b.bs + p % b.bs] = True
    b.k[~used.cuda()] = 0x7F
    b.v[~used.cuda()] = 0xFF
    got = b.call(jet)
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


@pytest.mark.parametrize("std", [1e-30, 0.0, 30.0, 1e30])
def test_query_range(jet, std):
    """Queries whose largest channel is far from one; a scale brings the scores back."""
    scale = None if std in (0.0, 30.0) else 0.05 / std
    Batch([(1, 100), (2, 33)], 4, 2, 128, 16, seed=7, q_std=std).check(jet, **({} if scale is None else dict(scale=scale)))


def test_a_dominant_key(jet):
    """One key far above the others, in the first, a middle and the last tile."""
    for at in (0, 150, 299):
        b = Batch([(1, 300)], 4, 1, 128, 16, seed=8 + at)
        slot = int(b.table[0, at // 16]) * 16 + at % 16
        b.k[slot, 0] = b.q[0, 0].float().mul(100).clamp(-448, 448).to(F8).view(U8)
        b.check(jet)


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("Hq,Hk", [(2, 2), (8, 2), (16, 1)])
@pytest.mark.parametrize("groups", [
    [(0, 6, 200)],                                   # everybody shares
    [(0, 2, 33), (2, 5, 128)],                       # two groups, one request alone
    [(1, 1, 50), (1, 4, 17), (4, 4, 9), (4, 6, 0)],  # empty groups, one without a prefix
    [(2, 6, 10 ** 6)],                               # longer than the first's length
    [(0, 3, -5), (3, 6, 1)]])
def test_shared_prefixes(jet, D, Hq, Hk, groups):
    """The prefix is read through the first request's row, whatever the others hold there."""
    Batch([(1, 230), (1, 201), (1, 256), (3, 300), (1, 40), (2, 221)], Hq, Hk, D, 16, seed=11,
          groups=groups).check(jet)


@pytest.mark.parametrize("n,prefix", [(70, 1), (40, 600), (200, 129)])
def test_large_groups(jet, n, prefix):
    b = Batch([(1, prefix + 1 + (7 * i) % 50) for i in range(n)], 8, 2, 128, 16, seed=n,
              groups=[(0, n, prefix)])
    b.check(jet)


def test_a_prefix_equals_no_prefix_where_the_tables_agree(jet):
    b = Batch([(1, 300), (1, 260), (2, 290)], 8, 2, 128, 16, seed=13, groups=[(0, 3, 256)])
    b.table[1:, :16] = b.table[0, :16]
    out, lse = b.check(jet)
    b.po = b.pl = None
    alone, lse1 = b.check(jet)
    assert (out.float() - alone.float()).abs().max() <= 2.0 ** -7 * alone.float().abs().max()


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("Hq,Hk", [(1, 1), (3, 1), (4, 2), (16, 2), (128, 1)])
@pytest.mark.parametrize("requests", [
    [(300, 300)], [(100, 1000), (256, 256), (1, 5), (64, 64)], [(513, 700)], [(40, 2000)], [(33, 33)] * 9])
def test_many_rows(jet, D, Hq, Hk, requests):
    """Units of up to 256 rows: of whole tokens, of one head's or of a request's."""
    Batch(requests, Hq, Hk, D, 16, seed=D + Hq + len(requests)).check(jet)


def test_many_rows_of_odd_batches(jet):
    """Lengths below the number of new tokens, of zero, tables without blocks, rows of no request."""
    b = Batch([(300, 300), (150, 600), (200, 200), (90, 90), (120, 400)], 8, 2, 128, 24, seed=31, behind=9)
    b.lengths[2], b.lengths[3] = 50, 0
    b.table[1, 3] = -1
    b.table[1, 7] = b.S // b.bs
    b.table[4] = -1
    b.lengths[0] = 100000                  # past the table's width
    b.check(jet)


@pytest.mark.parametrize("groups", [[(0, 3, 500)], [(0, 2, 100), (2, 4, 700)], [(1, 3, 333)], [(0, 4, 0)]])
def test_many_rows_behind_a_shared_prefix(jet, groups):
    Batch([(200, 900), (64, 600), (300, 1000), (7, 900)], 8, 2, 128, 16, seed=33, groups=groups).check(jet)


def test_maxima_that_keep_growing(jet):
    """Scores rise by far more than 2^8 from tile to tile, and fall again."""
    for rising in (True, False):
        b = Batch([(300, 1500)], 4, 1, 128, 16, seed=35)
        at = torch.arange(1500).cuda()
        slot = b.table[0].long()[at // 16] * 16 + at % 16
        size = (at if rising else 1499 - at).float() / 1500 * 400
        b.k[slot, 0] = (size[:, None] * torch.sign(b.q[299, 0].float())).to(F8).view(U8)
        b.check(jet)


def test_nan_behind_the_length_does_not_show_in_many_rows(jet):
    b = Batch([(100, 137), (200, 330)], 4, 2, 128, 64, seed=37, groups=[(0, 2, 100)])
    want = b.call(jet)
    used = torch.zeros((b.S,), dtype=torch.bool)
    for r, l in enumerate(b.lengths.tolist()):
        for p in range(l):
            used[int(b.table[r, p // b.bs]) * b.bs + p % b.bs] = True
    b.k[~used.cuda()] = 0x7F
    b.v[~used.cuda()] = 0xFF
    got = b.call(jet)
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("n,length", [(9, 77), (300, 300), (70, 333), (33, 4000)])
@pytest.mark.parametrize("prefix", [0, 1, 2])  # no group, a prefix before the key, one with it
def test_nan_in_a_later_key(jet, D, n, length, prefix):
    """NaN codes of a token in the middle of a chunk reach the queries from it on, none before,
    and another request's only where they are its prefix too."""
    at = length - n // 2 - 1                    # the position of the chunk's token n - n // 2 - 1
    shared = [None, min(length // 3, at), at + 3][prefix]
    b = Batch([(n, length), (2, length + 5)], 8, 2, D, 16, seed=41, groups=[(0, 2, shared)] if prefix else ())
    want, want_lse = b.call(jet)
    slot = int(b.table[0, at // b.bs]) * b.bs + at % b.bs
    before = n - n // 2 - 1
    for cache, code, sees in ((b.v, 0x7F, "value"), (b.k, 0xFF, "key")):
        kept = cache[slot].clone()
        cache[slot, 1, 17] = code
        got, lse = b.call(jet)
        assert torch.equal(got[:before], want[:before]) and torch.equal(lse[:before], want_lse[:before])
        if prefix < 2:
            assert torch.equal(got[n:], want[n:]) and torch.equal(lse[n:], want_lse[n:])
        else:
            assert torch.equal(got[n:, :4], want[n:, :4]) and got[n:, 4:, 17].isnan().all()
        assert torch.equal(got[before:n, :4], want[before:n, :4])           # the other head's
        assert got[before:n, 4:, 17].isnan().all()
        if sees == "key":
            assert lse[before:n, 4:].isnan().all() and got[before:n, 4:].isnan().all()
        else:
            assert torch.equal(lse[before:n], want_lse[before:n])
        cache[slot] = kept


def test_long_context(jet):
    """Many pieces of one unit."""
    g = torch.Generator().manual_seed(1)
    L, bs = 20001, 64
    b = Batch([(1, L)], 8, 2, 128, bs, seed=17)
    out, lse = b.call(jet)
    at = b.table[0].long()[torch.arange(L).cuda() // bs] * bs + torch.arange(L).cuda() % bs
    k, v = (c[at].view(F8).double() * s.double()[:, None] for c, s in ((b.k, b.ks), (b.v, b.vs)))
    x = torch.einsum("hgd,lhd->hgl", b.q[0].double().unflatten(0, (2, 4)), k) * 128 ** -0.5
    w = torch.softmax(x, -1)
    ref = torch.einsum("hgl,lhd->hgd", w, v).flatten(0, 1)
    mag = torch.einsum("hgl,lhd->hgd", w, v.abs()).flatten(0, 1)
    # as in Batch.reference; the scores stay below 8 in size, q . k below 2^11 of their units
    assert ((out[0].double() - ref).abs() <= 2.0 ** -8 * ref.abs() + 2.0 ** -9 * mag).all()
    assert ((lse[0].double() - torch.logsumexp(x, -1).flatten()).abs() <= 2.0 ** -11).all()


def test_the_same_bits_again_on_another_stream_and_in_a_graph(jet):
    b = Batch([(1, 230), (5, 201), (1, 256), (3, 300)], 8, 2, 128, 16, seed=19, groups=[(0, 3, 100)])
    want = b.call(jet)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    for _ in range(2):
        got = b.call(jet, stream=side)
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    out, lse = torch.zeros_like(want[0]), torch.zeros_like(want[1])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        jet.jet_kv_attention(b.q, b.k, b.v, b.ks, b.vs, b.table, b.bs, b.offsets, b.lengths, out, lse,
                             b.po, b.pl)
    for shorter in (0, 60):                # the replay takes the lengths as they are then
        b.lengths -= shorter
        graph.replay()
        torch.cuda.synchronize()
        want = b.call(jet)
        end = int(b.offsets[-1])
        assert torch.equal(out[:end], want[0][:end]) and torch.equal(lse[:end], want[1][:end])


def test_output_in_a_strided_tensor_and_the_allocating_form(jet):
    b = Batch([(1, 90), (2, 33)], 4, 2, 128, 16, seed=23, behind=2)
    want, lse = b.call(jet)
    rows = torch.zeros((b.T, 4 * 128 + 64), dtype=BF16, device="cuda")
    jet.jet_kv_attention(b.q, b.k, b.v, b.ks, b.vs, b.table, b.bs, b.offsets, b.lengths,
                         rows[:, :512].unflatten(1, (4, 128)))
    assert torch.equal(rows[:3, :512].unflatten(1, (4, 128)), want[:3]) and not rows[3:].any()
    assert not rows[:, 512:].any()
    got, gl = jet.kv_attention(b.q, b.k, b.v, b.ks, b.vs, b.table, b.bs, b.offsets, b.lengths, with_lse=True)
    assert torch.equal(got[:3], want[:3]) and torch.equal(gl[:3], lse[:3])
    assert not got[3:].any() and (gl[3:] == -INF).all()


def test_nothing_to_do(jet):
    b = Batch([(1, 9)], 2, 1, 64, 16)
    e = lambda *s, d=BF16: torch.empty(s, dtype=d, device="cuda")
    jet.jet_kv_attention(b.q[:0], b.k, b.v, b.ks, b.vs, b.table, 16, torch.tensor([0, 0]).cuda(), b.lengths,
                         e(0, 2, 64))
    out = torch.full((1, 2, 64), 7.0, dtype=BF16, device="cuda")
    jet.jet_kv_attention(b.q, b.k, b.v, b.ks, b.vs, b.table[:0], 16, torch.tensor([0]).cuda(),
                         b.lengths[:0], out)
    torch.cuda.synchronize()
    assert (out == 7).all()


def test_no_wait_ran_out(jet):
    code, word = jet.device_status()
    assert code == 0, hex(word)
