"""The softmax-attention operators at the ends of their ranges, and what their
outputs must not depend on."""
import math
import threading

import pytest
import torch

import attnref as ref
import linear_attention_recurrent_int8_b200 as lq
import test_gpu_attention as base
from test_gpu_attention import BF, DT, F32, Paged, check_attention, gen, no_device_errors, randn

pytestmark = pytest.mark.gpu


def split_of(io):
    """Relative rounding of the prefill's softmax weights."""
    return 2.0 ** -8 if io == BF else 0.0


# ------------------------------------------------------------------ score caps

# A cap as small as the header allows under a large scale: scale / cap to the
# 7th power is past FP32, scale / cap itself is not.
@pytest.mark.parametrize("io,D", [(BF, 64), (BF, 128), (BF, 256), (F32, 64)])
@pytest.mark.parametrize("scale,softcap", [(1e3, 1e-3), (-1e6, 1e-3), (1e6, 1.0)])
@pytest.mark.parametrize("size", [0.0, 1e-5, 1.0])
def test_small_caps_under_large_scales(io, D, scale, softcap, size):
    """Queries of zeros give the mean of the values, tiny and ordinary ones
    the capped softmax."""
    g = gen(61 + D)
    cfg = lq.AttnConfig(4, 2, D, io_dtype=io, scale=scale, softcap=softcap)
    n = 150
    pg = Paged(g, cfg, 2, 16, 10)
    # (powers of two in one channel: the scores' own rounding, which such a
    # scale brings up to the size of the cap, is none)
    pg.fill(g, [n, n])
    p = torch.arange(n, device="cuda")
    for b in range(2):
        at = (pg.table[b].long()[p // 16], slice(None), p % 16)
        k = torch.zeros(n, 2, D, dtype=DT[io], device="cuda")
        k[..., 0] = torch.exp2(torch.randint(-3, 4, (n, 2), generator=g, device="cuda").float()).to(DT[io])
        pg.k[at] = k
    q = torch.zeros(40, 4, D, dtype=DT[io], device="cuda")
    q[..., 0] = size * randn(g, 40, 4, dtype=DT[io])
    o = torch.empty_like(q)
    lq.lq_attn_prefill(cfg, pg.cache, torch.full((2,), n - 20, dtype=torch.int32, device="cuda"), None, q, o)
    od = torch.empty(2, 4, D, dtype=DT[io], device="cuda")
    lq.lq_attn_decode(cfg, pg.cache, torch.full((2,), n - 1, dtype=torch.int32, device="cuda"), q[:2].contiguous(), od)
    for b in range(2):
        rows = slice(20 * b, 20 * b + 20)
        # one product a score: its rounding, that of scale / cap and of their
        # product move y = s / cap by 3 half steps, so a score by at most
        # cap |y| (1 - tanh^2 y) 3 2^-24 < 2 cap 2^-24, inside the bound's 8
        check_exact_scores(cfg, pg, q[rows], o[rows], b, n - 20, split_of(io))
        check_exact_scores(cfg, pg, q[b:b + 1], od[b:b + 1], b, n - 1, 2.0 ** -17 if io == BF else 0.0)
    no_device_errors()


def check_exact_scores(cfg, pg, q, o, b, p0, split):
    """check_attention for scores that are single products: no error but the cap's."""
    n = q.shape[0]
    K, V = pg.dense(b, p0 + n)
    mask = torch.arange(p0 + n, device="cuda")[None] <= p0 + torch.arange(n, device="cuda")[:, None]
    for h in range(cfg.q_heads):
        kv = h // (cfg.q_heads // cfg.kv_heads)
        want, av, mag = ref.attend(q[:, h].double(), K[kv], V[kv], mask, cfg.c().scale, cfg.c().softcap)
        bound = ref.attend_bound(want, av, 0 * mag, cfg.head_dim, p0 + n, o.dtype, cfg.softcap, split)
        # the cap's polynomial: 5.6e-6 of the cap where it is used
        bound = bound + 2 * 5.6e-6 * min(cfg.softcap, 100.0) * av
        base.within(o[:, h], want, bound, f"{b} head {h}")


# (scale, cap, score over cap): scale / cap down to 1e-10, where its powers
# leave FP32, and caps of 300 and more, of which 5.6e-6 nears or passes the
# weights' rounding.
FAR_CAPS = [(1e-4, 1e6, 0.5), (1e-2, 1e6, 0.7), (0.3, 1e4, 0.6), (1e-3, 1e3, 0.5), (0.125, 50.0, 0.7), (1e-6, 50.0, 0.5)]
LARGE_CAPS = [(0.125, s, y) for s in (300.0, 1e3) for y in (0.3, 0.5, 0.7)] + \
    [(scale, s, y) for scale, s in ((2.0, 1e4), (20.0, 1e5), (200.0, 1e6)) for y in (0.1, 0.3, 0.5, 0.7)]


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("scale,softcap,y", FAR_CAPS + LARGE_CAPS)
def test_equal_capped_scores_weigh_the_same(D, scale, softcap, y):
    """Two tokens with the same key, opposite values and by far the largest
    score cancel, also where one stands in a tile with a score outside the
    reach of the cap's polynomial (far on the other side, without weight)."""
    g = gen(63)
    cfg = lq.AttnConfig(2, 1, D, scale=scale, softcap=softcap)
    n, new = 400, 3
    pg = Paged(g, cfg, 1, 16, 25)
    pg.fill(g, [n])
    pg.k.zero_()
    qk = y * softcap / scale  # the product of query and key
    k0 = 2.0 ** (math.floor(math.log2(qk)) // 2)
    q = torch.zeros(new, 2, D, dtype=torch.bfloat16, device="cuda")
    q[..., 0] = qk / k0

    def put(t, k, v):
        page = pg.table[0, t // 16].long()
        pg.k[page, 0, t % 16, 0] = k
        if v is not None:
            pg.v[page, 0, t % 16] = v
    v = randn(g, D, dtype=torch.bfloat16)
    put(5, k0, v)
    put(300, k0, -v)
    put(310, -3 * k0, None)
    o = torch.empty_like(q)
    lq.lq_attn_prefill(cfg, pg.cache, torch.full((1,), n - new, dtype=torch.int32, device="cuda"), None, q, o)
    # Equal products give equal scores where one formula serves both tokens.
    # Up to a cap of 100 a tile may take the polynomial: its error moves the
    # weights by 5.6e-6 cap, and they are rounded to 2^-8 of that difference's
    # neighbourhood of 1.  The other tokens weigh at most n e^(-cap tanh y).
    rest = n * math.exp(-softcap * math.tanh(0.99 * y))
    slack = 5.6e-6 * softcap + 2.0 ** -8 if softcap <= 100.0 else 2.0 ** -22
    bound = (0.5 * slack + 4 * rest) * v.double().abs() + rest * 10
    assert (o.double().abs() <= bound).all(), f"{o.double().abs().max().item():.2e}"
    no_device_errors()


# ------------------------------------------------------------------ what an output must not depend on

INDEPENDENT = [
    # new tokens, starts, Hq, Hkv, D, page, window, softcap, io
    ([5, 37, 130], [0, 211, 7], 4, 1, 64, 16, 0, 20.0, BF),
    ([5, 37, 130], [0, 211, 7], 4, 2, 128, 64, 0, 20.0, BF),
    ([5, 37, 130], [3, 211, 70], 2, 2, 256, 32, 50, 20.0, BF),
    ([5, 37, 130], [3, 211, 70], 8, 1, 64, 256, 70, 20.0, BF),
    ([5, 37, 130], [0, 211, 7], 4, 2, 128, 64, 33, 0.0, BF),
    ([3, 2, 5], [5000, 3, 900], 8, 2, 128, 128, 0, 20.0, BF),
    ([3, 2, 5], [5000, 3, 900], 4, 2, 64, 32, 700, 20.0, BF),
    ([5, 37, 130], [0, 211, 7], 4, 1, 64, 16, 0, 20.0, F32),
    ([5, 37, 130], [0, 211, 7], 3, 3, 128, 64, 0, 0.0, F32),
    ([5, 37, 130], [3, 211, 70], 8, 2, 256, 32, 50, 0.0, F32),
    ([3, 2, 5], [5000, 3, 900], 8, 2, 128, 128, 0, 20.0, F32),
]


class Independent:
    """A prefill call whose cache, queries and single places can be changed."""

    def __init__(self, new, start, Hq, Hkv, D, page, window, softcap, io):
        g = self.g = gen(71 + D)
        self.cfg = lq.AttnConfig(Hq, Hkv, D, io_dtype=io, window=window, softcap=softcap, scale=D ** -0.5)
        self.new, self.start = new, start
        reach = [s + n for s, n in zip(start, new)]
        self.pg = Paged(g, self.cfg, len(new), page, -(-max(reach) // page) + 1)
        self.pg.fill(g, reach)
        self.cu = torch.tensor([0] + torch.tensor(new).cumsum(0).tolist(), dtype=torch.int32, device="cuda")
        self.pos = torch.tensor(start, dtype=torch.int32, device="cuda")
        self.q = randn(g, sum(new), Hq, D, dtype=DT[io], scale=2.0)
        # places of the cache that some new token of their sequence sees
        self.seen = torch.zeros(self.pg.k.shape[:1] + self.pg.k.shape[2:3], dtype=torch.bool, device="cuda")
        for b, (n, s) in enumerate(zip(new, start)):
            p = torch.arange(max(0, s + 1 - window) if window else 0, s + n, device="cuda")
            self.seen[self.pg.table[b].long()[p // page], p % page] = True
        self.seen = self.seen[:, None, :, None].expand_as(self.pg.k)

    def run(self):
        o = torch.empty_like(self.q)
        lq.lq_attn_prefill(self.cfg, self.pg.cache, self.pos, self.cu, self.q, o)
        return o

    def decode(self):
        """The last new token of each sequence."""
        q = self.q[self.cu[1:].long() - 1].contiguous()
        o = torch.empty_like(q)
        lq.lq_attn_decode(self.cfg, self.pg.cache, self.pos + torch.tensor(self.new, device="cuda", dtype=torch.int32) - 1, q, o)
        return o


ANYTHING = [math.nan, 3e38, -3e38, math.inf, 7.0]


@pytest.mark.parametrize("case", INDEPENDENT)
def test_outputs_do_not_depend_on_places_that_no_token_sees(case):
    c = Independent(*case)
    for x in (c.pg.k, c.pg.v):
        x[~c.seen] = 0.0
    want, want_d = c.run(), c.decode()
    for b, s in enumerate(c.start):
        rows = slice(int(c.cu[b]), int(c.cu[b + 1]))
        check_attention(c.cfg, c.pg, c.q[rows], want[rows], b, s, split_of(c.cfg.io_dtype), f"sequence {b}")
    for fill in ANYTHING:
        for x in (c.pg.k, c.pg.v):
            x[~c.seen] = fill
        assert torch.equal(c.run(), want), f"prefill: {fill} in places that no token sees"
        assert torch.equal(c.decode(), want_d), f"decode: {fill} in places that no token sees"
    no_device_errors()


@pytest.mark.parametrize("case", INDEPENDENT)
def test_outputs_do_not_depend_on_later_tokens(case):
    """Another key, value and query of a sequence's last new token leave the
    outputs of those before it as they are, to the bit."""
    c = Independent(*case)
    want = c.run()
    last = (c.cu[1:] - 1).long()
    before = torch.ones(c.q.shape[0], dtype=torch.bool, device="cuda")
    before[last] = False
    page = c.pg.page
    for size in (30.0, 3000.0, 1e-3):
        for b, (n, s) in enumerate(zip(c.new, c.start)):
            p = s + n - 1
            at = (c.pg.table[b, p // page].long(), slice(None), p % page)
            for x in (c.pg.k, c.pg.v):
                x[at] = randn(c.g, *x[at].shape, dtype=x.dtype, scale=size)
        c.q[last] = randn(c.g, *c.q[last].shape, dtype=c.q.dtype, scale=size)
        assert torch.equal(c.run()[before], want[before]), f"size {size}"
    # infinite keys and queries (a value that a row does not see has to be finite)
    for b, (n, s) in enumerate(zip(c.new, c.start)):
        p = s + n - 1
        c.pg.k[c.pg.table[b, p // page].long(), :, p % page, ::3] = math.inf
        c.pg.v[c.pg.table[b, p // page].long(), :, p % page] = 0.5
    c.q[last, :, 1::5] = -math.inf
    assert torch.equal(c.run()[before], want[before]), "infinite"
    no_device_errors()


@pytest.mark.parametrize("Hq,Hkv,D,io", [(4, 1, 64, F32), (20, 2, 128, F32), (6, 2, 256, F32), (8, 1, 128, BF), (40, 2, 64, BF)])
def test_heads_do_not_depend_on_each_other(Hq, Hkv, D, io):
    """Infinite or NaN queries of one head leave the outputs of the others as
    they are, to the bit."""
    g = gen(73)
    cfg = lq.AttnConfig(Hq, Hkv, D, io_dtype=io)
    lens = [777, 1, 3000]
    pg = Paged(g, cfg, 3, 32, 100)
    pg.fill(g, lens)
    q = randn(g, 3, Hq, D, dtype=DT[io], scale=2.0)
    pos = torch.tensor(lens, dtype=torch.int32, device="cuda") - 1

    def run():
        od, op = torch.empty_like(q), torch.empty_like(q)
        lq.lq_attn_decode(cfg, pg.cache, pos, q, od)
        lq.lq_attn_prefill(cfg, pg.cache, pos, None, q, op)
        return od, op
    want = run()
    for h in range(Hq):
        others = torch.arange(Hq, device="cuda") != h
        keep = q[:, h].clone()
        for x in (math.inf, math.nan):
            q[:, h, 3::7] = x
            for got, w in zip(run(), want):
                assert torch.equal(got[:, others], w[:, others]), f"head {h}, {x}"
        q[:, h] = keep
    no_device_errors()


@pytest.mark.parametrize("case", INDEPENDENT)
def test_outputs_do_not_depend_on_other_sequences(case):
    """Other queries, keys and values of one sequence, NaN among them, leave
    the outputs of the others as they are, to the bit."""
    c = Independent(*case)
    want = c.run()
    for b in range(len(c.new)):
        rows = torch.zeros(c.q.shape[0], dtype=torch.bool, device="cuda")
        rows[int(c.cu[b]):int(c.cu[b + 1])] = True
        q, pages = c.q.clone(), c.pg.table[b].long()
        k, v = c.pg.k[pages].clone(), c.pg.v[pages].clone()
        for size in (1e-3, 3000.0, math.nan):
            c.q[rows] = randn(c.g, *c.q[rows].shape, dtype=c.q.dtype, scale=size)
            c.pg.k[pages] = randn(c.g, *k.shape, dtype=k.dtype, scale=size)
            c.pg.v[pages] = randn(c.g, *v.shape, dtype=v.dtype, scale=size)
            assert torch.equal(c.run()[~rows], want[~rows]), f"sequence {b}, size {size}"
        c.q.copy_(q)
        c.pg.k[pages], c.pg.v[pages] = k, v
    no_device_errors()


# ------------------------------------------------------------------ every key once

def check_weights_of_pages(cfg, pg, o, b, p0):
    """Outputs for queries of zeros over values that are 1 in one channel, by
    the token's group of 16: channel c is the share of the visible tokens whose
    group is c modulo the head size.  Weights of 1, sums of whole numbers and a
    power of two per part are exact, so the reciprocal of the sum (2 half steps
    of FP32), a product and the output's rounding are all the error there is:
    one token more or less in a group, or a group left out, is far above it."""
    n = o.shape[0]
    for i in range(n):
        p = p0 + i
        lo = max(0, p + 1 - cfg.window) if cfg.window else 0
        t = torch.arange(lo, p + 1, device="cuda")
        want = torch.bincount(t // 16 % cfg.head_dim, minlength=cfg.head_dim).double() / len(t)
        bound = (ref.HALF[o.dtype] + 4 * 2.0 ** -24) * want
        base.within(o[i], want.expand(cfg.q_heads, -1), bound, f"sequence {b}, position {p}")


def pages_by_group(cfg, g, lens, page):
    """A cache whose values are the groups' indicators; keys are random."""
    pg = Paged(g, cfg, len(lens), page, -(-max(lens) // page))
    pg.fill(g, lens)
    for b, n in enumerate(lens):
        t = torch.arange(n, device="cuda")
        v = torch.zeros(n, cfg.kv_heads, cfg.head_dim, dtype=cfg.io_torch_dtype, device="cuda")
        v[t, :, t // 16 % cfg.head_dim] = 1.0
        pg.v[pg.table[b].long()[t // page], :, t % page] = v
    return pg


@pytest.mark.parametrize("io", [BF, F32])
@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("new,start,Hq,Hkv,page,window", [
    # one sequence: the keys of a tile split over up to 8 blocks
    ([1], [127], 2, 1, 16, 0), ([1], [128], 2, 1, 16, 0), ([2], [255], 2, 1, 64, 0), ([1], [320], 4, 1, 16, 0),
    ([3], [511], 2, 1, 32, 0), ([2], [1022], 8, 2, 16, 0), ([5], [2000], 2, 2, 128, 0), ([2], [5119], 4, 1, 256, 0),
    ([3], [20011], 4, 2, 64, 0), ([2], [6000], 2, 1, 16, 1000), ([4], [6000], 2, 1, 32, 4097),
    # several, of very different lengths
    ([1, 3, 2], [9000, 17, 300], 2, 1, 16, 0), ([2, 1, 4, 1], [700, 0, 1300, 260], 4, 4, 64, 0),
    ([4, 9], [3000, 130], 2, 1, 32, 129),
    # longer runs: tiles of many rows
    ([70, 33], [200, 1000], 8, 1, 64, 0), ([300], [77], 4, 1, 16, 100),
])
def test_prefill_takes_every_key_once(new, start, Hq, Hkv, page, window, D, io):
    g = gen(81)
    cfg = lq.AttnConfig(Hq, Hkv, D, io_dtype=io, window=window)
    lens = [s + n for s, n in zip(start, new)]
    pg = pages_by_group(cfg, g, lens, page)
    cu = torch.tensor([0] + torch.tensor(new).cumsum(0).tolist(), dtype=torch.int32, device="cuda")
    q = torch.zeros(sum(new), Hq, D, dtype=DT[io], device="cuda")
    o = torch.full_like(q, 3.0)
    lq.lq_attn_prefill(cfg, pg.cache, torch.tensor(start, dtype=torch.int32, device="cuda"), cu, q, o)
    for b, s in enumerate(start):
        check_weights_of_pages(cfg, pg, o[int(cu[b]):int(cu[b + 1])], b, s)
    no_device_errors()


@pytest.mark.parametrize("io", [BF, F32])
@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("lens,Hq,Hkv,page,window", [
    ([1, 15, 16, 17, 31, 32, 33, 500], 2, 1, 16, 0),
    ([1, 15, 16, 17, 31, 32, 33, 500], 6, 2, 32, 17),
    ([20011], 4, 2, 64, 0), ([6000, 1, 900], 2, 2, 16, 1000),
    ([2500, 40], 24, 1, 128, 0), ([3000, 800, 17], 40, 1, 16, 0), ([900, 2000], 33, 1, 64, 700),
])
def test_decode_takes_every_key_once(lens, Hq, Hkv, page, window, D, io):
    g = gen(82)
    cfg = lq.AttnConfig(Hq, Hkv, D, io_dtype=io, window=window)
    pg = pages_by_group(cfg, g, lens, page)
    q = torch.zeros(len(lens), Hq, D, dtype=DT[io], device="cuda")
    o = torch.full_like(q, 3.0)
    lq.lq_attn_decode(cfg, pg.cache, torch.tensor(lens, dtype=torch.int32, device="cuda") - 1, q, o)
    for b, n in enumerate(lens):
        check_weights_of_pages(cfg, pg, o[b:b + 1], b, n - 1)
    no_device_errors()


# ------------------------------------------------------------------ decode: row groups and joins

@pytest.mark.parametrize("pos,Hq,Hkv,D,page,window,softcap,io", [
    # FP32 with 2 and 3 row groups of 8 to a key-value head, BF16 with 3 of 16
    ([900, 17, 401], 16, 1, 128, 16, 0, 0.0, F32),
    ([900, 17, -1, 401], 40, 2, 64, 32, 0, 0.0, F32),
    ([900, 17, 401], 20, 1, 256, 64, 100, 20.0, F32),
    ([900, 17, 401], 40, 1, 128, 16, 0, 0.0, BF),
    ([5000, 0], 33, 1, 64, 64, 0, 0.0, BF),
    ([30000, 12], 80, 2, 256, 128, 0, 30.0, BF),
    ([30000], 20, 1, 64, 16, 0, 0.0, F32),
    # more row groups than warps of a block
    ([700, 90], 160, 1, 64, 16, 0, 0.0, BF),
    ([700, 90], 100, 1, 128, 16, 0, 0.0, F32),
])
def test_decode_row_groups(pos, Hq, Hkv, D, page, window, softcap, io):
    base.test_decode(pos, Hq, Hkv, D, page, window, softcap, io)


@pytest.mark.parametrize("D,Hkv,io", [(64, 2, BF), (128, 1, BF), (256, 2, BF), (64, 2, F32), (128, 4, F32)])
def test_decode_of_few_long_among_many_short_sequences(D, Hkv, io):
    """Enough heads for blocks that join 8 of them, some with more parts than a
    warp joins alone."""
    g = gen(83)
    pos = torch.randint(-1, 100, (60,), generator=g, device="cuda").tolist()
    pos[7], pos[44] = 30000, 17011
    base.test_decode(pos, 32, Hkv, D, 64, 0, 0.0, io)


# ------------------------------------------------------------------ calls at once

def test_graphs_at_once_and_calls_from_threads():
    """A layer's step of several configurations: graphs of it replayed at once
    on streams of their own, and calls from as many host threads, give what
    the calls give alone (workspaces allocated by the calls)."""
    steps, outs, streams = [], [], []
    for i, (D, io) in enumerate([(64, BF), (128, BF), (256, BF), (64, F32), (128, F32), (256, F32), (64, BF)]):
        g = gen(90 + i)
        cfg = lq.AttnConfig(8, 2, D, io_dtype=io, norm=lq.LQ_NORM_RMS, rot_dim=D // 2, softcap=30.0 if i % 2 else 0.0)
        pg = Paged(g, cfg, 3, 64, 40)
        pg.fill(g, [2001, 4, 701])
        pos = torch.tensor([2000, 3, 700], dtype=torch.int32, device="cuda")
        qkv = randn(g, 3, 12 * D, dtype=DT[io])
        w, cs = 1 + 0.2 * randn(g, D), ref.table(D // 2, 40 * 64).cuda()
        qo, od, op = (torch.zeros(3, 8, D, dtype=DT[io], device="cuda") for _ in range(3))

        def step(cfg=cfg, pg=pg, pos=pos, qkv=qkv, w=w, cs=cs, qo=qo, od=od, op=op, D=D):
            q, k, v = (qkv[:, a * D:b * D].view(3, -1, D) for a, b in ((0, 8), (8, 10), (10, 12)))
            lq.lq_kv_append(cfg, pg.cache, pos, None, q, k, v, w, w, cs, qo)
            lq.lq_attn_decode(cfg, pg.cache, pos, qo, od)
            lq.lq_attn_prefill(cfg, pg.cache, pos, None, qo, op)
        steps.append(step)
        outs.append((qo, od, op))
        streams.append(torch.cuda.Stream())
    for step in steps:
        step()
    torch.cuda.synchronize()
    alone = [[x.clone() for x in xs] for xs in outs]

    def check(what):
        torch.cuda.synchronize()
        for i, (xs, ys) in enumerate(zip(outs, alone)):
            assert all(torch.equal(x, y) for x, y in zip(xs, ys)), f"{what}, configuration {i}"
            for x in xs:
                x.zero_()
        torch.cuda.synchronize()

    check("alone")
    graphs = [torch.cuda.CUDAGraph() for _ in steps]
    for graph, step in zip(graphs, steps):
        with torch.cuda.graph(graph):
            step()
    for _ in range(20):
        for graph, stream in zip(graphs, streams):
            with torch.cuda.stream(stream):
                graph.replay()
    check("graphs at once")
    failed = []

    def work(step, stream):
        try:
            with torch.cuda.stream(stream):
                for _ in range(50):
                    step()
        except Exception as e:  # for the assertion below: a thread's exception ends nothing else
            failed.append(e)
    threads = [threading.Thread(target=work, args=a) for a in zip(steps, streams)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not failed, failed
    check("threads")
    no_device_errors()
