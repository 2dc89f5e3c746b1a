"""The softmax-attention operators against plain 64-bit implementations."""
import math

import pytest
import torch

import attnref as ref
import linear_attention_recurrent_int8_b200 as lq

pytestmark = pytest.mark.gpu

DT = {lq.LQ_BF16: torch.bfloat16, lq.LQ_F32: torch.float32}
BF, F32 = lq.LQ_BF16, lq.LQ_F32


def gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def randn(g, *shape, dtype=torch.float32, scale=1.0):
    return (torch.randn(*shape, generator=g, device="cuda") * scale).to(dtype)


def within(got, want, bound, what):
    assert torch.isfinite(got.double()).all(), what
    if got.numel() == 0:
        return
    over = (got.double() - want).abs() - bound
    assert over.max().item() <= 0, f"{what}: {over.max().item():.3e} over the bound"


def no_device_errors():
    assert lq.lq_device_errors() == 0


# ------------------------------------------------------------------ norm and rotation

NORM_CASES = [
    # T, Hq, Hkv, D, norm, weights, rot, pairs, io
    (1, 1, 1, 64, lq.LQ_NORM_L2, False, 0, 0, BF),
    (1, 32, 8, 128, lq.LQ_NORM_RMS, True, 128, lq.LQ_ROT_HALVES, BF),
    (7, 6, 3, 64, lq.LQ_NORM_RMS, True, 64, lq.LQ_ROT_ADJACENT, BF),
    (130, 12, 4, 128, lq.LQ_NORM_L2, False, 48, lq.LQ_ROT_HALVES, F32),
    (33, 5, 5, 256, lq.LQ_NORM_RMS, True, 64, lq.LQ_ROT_HALVES, BF),
    (33, 5, 1, 256, lq.LQ_NORM_RMS, True, 256, lq.LQ_ROT_HALVES, F32),
    (19, 16, 2, 256, lq.LQ_NORM_NONE, False, 16, lq.LQ_ROT_ADJACENT, F32),
    (3001, 32, 32, 128, lq.LQ_NORM_L2, True, 0, 0, BF),
    (2500, 24, 8, 64, lq.LQ_NORM_RMS, True, 32, lq.LQ_ROT_HALVES, F32),
    (2500, 24, 8, 64, lq.LQ_NORM_NONE, False, 64, lq.LQ_ROT_ADJACENT, BF),
]


@pytest.mark.parametrize("T,Hq,Hkv,D,norm,weights,rot,pairs,io", NORM_CASES)
def test_norm_rotate(T, Hq, Hkv, D, norm, weights, rot, pairs, io):
    g = gen(T + D)
    dt = DT[io]
    cfg = lq.AttnConfig(Hq, Hkv, D, io_dtype=io, norm=norm, rot_dim=rot, rot_pairs=pairs)
    qk = randn(g, T, (Hq + Hkv) * D + 16, dtype=dt, scale=5.0)
    q, k = qk[:, :Hq * D].view(T, Hq, D), qk[:, Hq * D:(Hq + Hkv) * D].view(T, Hkv, D)
    if T > 2:
        q[2] = 0  # a row of zeros stays zero
    pos = torch.randint(0, 70000, (T,), generator=g, device="cuda", dtype=torch.int32)
    if T > 4:
        pos[4] = -1
        pos[T - 1] = -7
    cs = ref.table(rot, 70000).cuda() if rot else None
    wq, wk = (1 + 0.3 * randn(g, D), 1 + 0.3 * randn(g, D)) if weights else (None, None)
    qo, ko = torch.full((T, Hq, D), 3.0, dtype=dt, device="cuda"), torch.full((T, Hkv, D), 3.0, dtype=dt, device="cuda")
    lq.lq_qk_norm_rotate(cfg, q, k, wq, wk, pos, cs, qo, ko)
    for x, w, out, name in ((q, wq, qo, "q"), (k, wk, ko, "k")):
        y, mag = ref.norm_rotate(x, norm, 1e-6, w, rot, pairs == lq.LQ_ROT_ADJACENT, cs, pos.clamp(min=0).long())
        live = pos >= 0
        within(out[live], y[live], ref.rows_bound(y, mag, dt)[live], name)
        assert (out[~live] == 3.0).all()
    # q alone, in place
    x = q.contiguous()
    lq.lq_qk_norm_rotate(cfg, x, None, wq, None, pos, cs, x, None)
    live = pos >= 0
    assert torch.equal(x[live], qo[live]) and torch.equal(x[~live], q[~live])
    no_device_errors()


def test_norm_rotate_without_positions_and_batched_shapes():
    """[B, n, H, D] slices as the linear-attention calls take them; no positions."""
    g = gen(5)
    B, n, H, D = 3, 9, 4, 128
    cfg = lq.AttnConfig(H, H, D, norm=lq.LQ_NORM_L2)
    qkv = randn(g, B, n, 3 * H * D, dtype=torch.bfloat16)
    q, k = (qkv[..., i * H * D:(i + 1) * H * D].unflatten(-1, (H, D)) for i in range(2))
    qo, ko = torch.empty(B, n, H, D, dtype=torch.bfloat16, device="cuda"), torch.empty(B, n, H, D, dtype=torch.bfloat16, device="cuda")
    lq.lq_qk_norm_rotate(cfg, q, k, None, None, None, None, qo, ko)
    for x, out in ((q, qo), (k, ko)):
        y, mag = ref.norm_rotate(x.reshape(-1, H, D), 1, 1e-6, None, 0, False, None, None)
        within(out.view(-1, H, D), y, ref.rows_bound(y, mag, torch.bfloat16), "norm")
    no_device_errors()


def test_positions_past_the_table_are_skipped_and_reported():
    g = gen(6)
    cfg = lq.AttnConfig(2, 1, 64, rot_dim=64)
    q, k = randn(g, 5, 2, 64, dtype=torch.bfloat16), randn(g, 5, 1, 64, dtype=torch.bfloat16)
    cs = ref.table(64, 10).cuda()
    pos = torch.tensor([0, 10, 9, -1, 1 << 30], dtype=torch.int32, device="cuda")
    qo, ko = torch.zeros_like(q), torch.zeros_like(k)
    lq.lq_qk_norm_rotate(cfg, q, k, None, None, pos, cs, qo, ko)
    assert lq.lq_device_errors() == lq.LQ_DEVERR_BAD_POSITION
    for t in (1, 3, 4):
        assert (qo[t] == 0).all() and (ko[t] == 0).all()
    for t in (0, 2):
        assert (qo[t] != 0).any() and (ko[t] != 0).any()


# ------------------------------------------------------------------ a paged cache

class Paged:
    """A cache with its pages in random order, every place not yet written NaN."""

    def __init__(self, g, cfg, B, page, width, spare=3):
        P = B * width + spare
        shape = (P, cfg.kv_heads, page, cfg.head_dim)
        self.k = torch.full(shape, math.nan, dtype=cfg.io_torch_dtype, device="cuda")
        self.v = torch.full(shape, math.nan, dtype=cfg.io_torch_dtype, device="cuda")
        order = torch.randperm(P, generator=g, device="cuda")[:B * width]
        self.table = order.view(B, width).to(torch.int32)
        self.page, self.cfg = page, cfg
        self.cache = lq.KvCache(cfg, self.k, self.v, self.table)

    def fill(self, g, lens, scale=1.0):
        """Random keys and values for the first lens[b] tokens of each sequence."""
        c = self.cfg
        for b, n in enumerate(lens):
            if n <= 0:
                continue
            p = torch.arange(n, device="cuda")
            at = (self.table[b].long()[p // self.page], slice(None), p % self.page)
            self.k[at] = randn(g, n, c.kv_heads, c.head_dim, dtype=c.io_torch_dtype, scale=scale)
            self.v[at] = randn(g, n, c.kv_heads, c.head_dim, dtype=c.io_torch_dtype)

    def dense(self, b, n):
        return tuple(ref.paged(x, self.table[b], self.page, n) for x in (self.k, self.v))


def check_attention(cfg, pg, q, o, b, p0, split, what):
    """Rows q, o [n, Hq, D] of sequence b at positions p0, p0 + 1, ..."""
    n = q.shape[0]
    K, V = pg.dense(b, p0 + n)
    G = cfg.q_heads // cfg.kv_heads
    pos = p0 + torch.arange(n, device="cuda")[:, None]
    j = torch.arange(p0 + n, device="cuda")[None]
    mask = j <= pos
    if cfg.window:
        mask &= j > pos - cfg.window
    scale = cfg.c().scale
    for h in range(cfg.q_heads):
        want, av, mag = ref.attend(q[:, h].double(), K[h // G], V[h // G], mask, scale, cfg.softcap)
        within(o[:, h], want, ref.attend_bound(want, av, mag, cfg.head_dim, p0 + n, o.dtype, cfg.softcap, split),
               f"{what} head {h}")


APPEND_CASES = [
    # new tokens per sequence (None: uniform), starts, Hq, Hkv, D, page, norm, rot, pairs, io
    ([1, 1, 1, 1], [0, -1, 15, 16], 4, 2, 64, 16, lq.LQ_NORM_RMS, 64, lq.LQ_ROT_HALVES, BF),
    ([3, 3, 3], [14, 0, 31], 6, 3, 128, 16, lq.LQ_NORM_L2, 32, lq.LQ_ROT_ADJACENT, F32),
    ([0, 5, 1, 0, 40, 0], [3, 0, 60, -1, 7, 0], 8, 1, 128, 32, lq.LQ_NORM_RMS, 128, lq.LQ_ROT_HALVES, BF),
    ([17, 0, 2], [0, 9, -1], 2, 2, 256, 64, lq.LQ_NORM_NONE, 16, lq.LQ_ROT_ADJACENT, BF),
    ([9, 130], [100, 0], 5, 5, 256, 128, lq.LQ_NORM_RMS, 0, 0, F32),
    ([700, 1, 350], [1, 0, 255], 24, 8, 64, 256, lq.LQ_NORM_NONE, 0, 0, BF),
]


@pytest.mark.parametrize("new,start,Hq,Hkv,D,page,norm,rot,pairs,io", APPEND_CASES)
@pytest.mark.parametrize("with_q", [True, False])
def test_append(new, start, Hq, Hkv, D, page, norm, rot, pairs, io, with_q):
    g = gen(len(new) + D)
    dt = DT[io]
    cfg = lq.AttnConfig(Hq, Hkv, D, io_dtype=io, norm=norm, rot_dim=rot, rot_pairs=pairs)
    B = len(new)
    reach = max(max(s, 0) + n for s, n in zip(start, new))
    pg = Paged(g, cfg, B, page, -(-reach // page))
    uniform = len(set(new)) == 1
    pad = 0 if uniform else 4
    T = sum(new) + pad
    cu = None
    if not uniform:
        cu = torch.tensor([0] + torch.tensor(new).cumsum(0).tolist(), dtype=torch.int32, device="cuda")
    qkv = randn(g, T, (Hq + 2 * Hkv) * D, dtype=dt, scale=2.0)
    q, k, v = (qkv[:, a * D:b * D].view(T, -1, D) for a, b in ((0, Hq), (Hq, Hq + Hkv), (Hq + Hkv, Hq + 2 * Hkv)))
    cs = ref.table(rot, reach).cuda() if rot else None
    w = (1 + 0.3 * randn(g, D), 1 + 0.3 * randn(g, D)) if norm == lq.LQ_NORM_RMS else (None, None)
    pos = torch.tensor(start, dtype=torch.int32, device="cuda")
    qo = torch.full((T, Hq, D), 3.0, dtype=dt, device="cuda") if with_q else None
    lq.lq_kv_append(cfg, pg.cache, pos, cu, q if with_q else None, k, v, w[0] if with_q else None, w[1], cs, qo)
    seen_k = torch.zeros(pg.k.shape[:3], dtype=torch.bool, device="cuda")
    row = 0
    for b, (n, s) in enumerate(zip(new, start)):
        rows = slice(row, row + n)
        row += n
        if s < 0:
            assert qo is None or (qo[rows] == 3.0).all()
            continue
        p = s + torch.arange(n, device="cuda")
        ids, off = pg.table[b].long()[p // page], p % page
        y, mag = ref.norm_rotate(k[rows], norm, 1e-6, w[1], rot, pairs == lq.LQ_ROT_ADJACENT, cs, p)
        within(pg.k[ids, :, off], y, ref.rows_bound(y, mag, dt), "k")
        assert torch.equal(pg.v[ids, :, off], v[rows])
        if with_q:
            y, mag = ref.norm_rotate(q[rows], norm, 1e-6, w[0], rot, pairs == lq.LQ_ROT_ADJACENT, cs, p)
            within(qo[rows], y, ref.rows_bound(y, mag, dt), "q")
        seen_k[ids, :, off] = True
    assert qo is None or (qo[row:] == 3.0).all()  # padding rows
    # everything else is as it was
    assert pg.k[~seen_k].isnan().all() and pg.v[~seen_k].isnan().all()
    no_device_errors()


def test_append_skips_and_reports_bad_places():
    g = gen(9)
    cfg = lq.AttnConfig(2, 1, 64, rot_dim=64)
    pg = Paged(g, cfg, 4, 16, 2)
    pg.table[1, 0] = pg.k.shape[0]  # not a page
    pg.table[2, 0] = -1
    k = randn(g, 4, 1, 64, dtype=torch.bfloat16)
    cs = ref.table(64, 64).cuda()
    pos = torch.tensor([3, 5, 5, 32], dtype=torch.int32, device="cuda")  # 32: past the block table
    lq.lq_kv_append(cfg, pg.cache, pos, None, None, k, k, None, None, cs, None)
    assert lq.lq_device_errors() == lq.LQ_DEVERR_BAD_PAGE | lq.LQ_DEVERR_BAD_POSITION
    assert (~pg.k.isnan()).sum() == 64 and (~pg.v.isnan()).sum() == 64
    assert torch.equal(pg.v[pg.table[0, 0].long(), 0, 3], k[0, 0])


# ------------------------------------------------------------------ decode

DECODE_CASES = [
    # positions, Hq, Hkv, D, page, window, softcap, io
    ([0], 1, 1, 64, 16, 0, 0.0, BF),
    ([0, 1, 14, 15, 16, 17, -1, 31, 32, 33], 4, 2, 64, 16, 0, 0.0, BF),
    ([0, 1, 14, 15, 16, 17, -1, 31, 32, 33], 4, 2, 128, 16, 0, 0.0, F32),
    ([5, 300, 63, 64, 65], 32, 8, 128, 64, 0, 0.0, BF),
    ([5, 300, 63, 64, 65], 7, 1, 256, 32, 0, 0.0, BF),
    ([5, 300, 63, 64, 65], 7, 1, 256, 32, 0, 0.0, F32),
    ([900, 17, 401], 9, 1, 128, 16, 0, 30.0, BF),
    ([900, 17, 401], 16, 1, 64, 128, 0, 0.0, BF),
    ([900, 17, 401], 40, 2, 64, 128, 37, 0.0, BF),
    ([900, 17, 401], 48, 2, 256, 256, 100, 20.0, BF),
    ([900, 17, 401], 16, 2, 64, 16, 1, 0.0, F32),
    ([900, 17, 401, 16, 15], 9, 3, 128, 16, 16, 5.0, F32),
    ([900, 17, 401, 16, 15], 6, 3, 128, 16, 17, 5.0, BF),
    ([40000, -1], 8, 1, 128, 64, 0, 0.0, BF),
    ([40000, 3], 2, 1, 64, 16, 0, 0.0, F32),
    ([30011], 3, 1, 256, 64, 0, 0.0, BF),
    ([30011], 3, 1, 256, 64, 0, 0.0, F32),
    ([-1, -5, -1], 4, 4, 128, 16, 0, 0.0, BF),
]


@pytest.mark.parametrize("pos,Hq,Hkv,D,page,window,softcap,io", DECODE_CASES)
def test_decode(pos, Hq, Hkv, D, page, window, softcap, io):
    g = gen(Hq + D)
    dt = DT[io]
    cfg = lq.AttnConfig(Hq, Hkv, D, io_dtype=io, window=window, softcap=softcap)
    B = len(pos)
    pg = Paged(g, cfg, B, page, max(max(pos), 0) // page + 1)
    pg.fill(g, [p + 1 for p in pos])
    q = randn(g, B, Hq, D, dtype=dt, scale=2.0)
    o = torch.full((B, Hq, D), 3.0, dtype=dt, device="cuda")
    lq.lq_attn_decode(cfg, pg.cache, torch.tensor(pos, dtype=torch.int32, device="cuda"), q, o)
    for b, p in enumerate(pos):
        if p < 0:
            assert (o[b] == 3.0).all()
        else:
            check_attention(cfg, pg, q[b:b + 1], o[b:b + 1], b, p, 2.0 ** -17 if io == BF else 0.0, f"sequence {b}")
    no_device_errors()


@pytest.mark.parametrize("io", [BF, F32])
def test_decode_many_sequences(io):
    """More sequences than threads of a block scan at once, mostly short or idle."""
    g = gen(77)
    cfg = lq.AttnConfig(2, 1, 64, io_dtype=io)
    B = 700
    pos = torch.randint(-1, 40, (B,), generator=g, device="cuda", dtype=torch.int32)
    pg = Paged(g, cfg, B, 16, 3)
    pl = pos.tolist()
    pg.fill(g, [p + 1 for p in pl])
    q = randn(g, B, 2, 64, dtype=DT[io], scale=2.0)
    o = torch.full((B, 2, 64), 3.0, dtype=DT[io], device="cuda")
    lq.lq_attn_decode(cfg, pg.cache, pos, q, o)
    for b in range(0, B, 7):
        if pl[b] < 0:
            assert (o[b] == 3.0).all()
        else:
            check_attention(cfg, pg, q[b:b + 1], o[b:b + 1], b, pl[b], 2.0 ** -17 if io == BF else 0.0, f"sequence {b}")
    no_device_errors()


@pytest.mark.parametrize("io,D", [(BF, 128), (BF, 256), (F32, 64)])
def test_decode_infinite_scores(io, D):
    """-inf scores weigh nothing, wherever they stand; a sequence of nothing
    else is NaN, as its formula; a NaN key or value makes its own sequence NaN only."""
    g = gen(3)
    cfg = lq.AttnConfig(2, 1, D, io_dtype=io)
    n = 3000
    pg = Paged(g, cfg, 4, 16, -(-n // 16))
    pg.fill(g, [n] * 4)
    q = torch.zeros(4, 2, D, dtype=DT[io], device="cuda")
    q[..., 0] = 1.0
    hit = torch.arange(n, device="cuda")
    gone = (hit < 2000) | (hit % 3 == 0)

    def put(b, t, x):
        pg.k[pg.table[b].long()[t // 16], 0, t % 16, 0] = x
    put(0, hit[gone], -math.inf)
    put(1, hit, -math.inf)
    put(2, hit[1234:1235], math.nan)
    o = torch.empty(4, 2, D, dtype=DT[io], device="cuda")
    lq.lq_attn_decode(cfg, pg.cache, torch.full((4,), n - 1, dtype=torch.int32, device="cuda"), q, o)
    K, V = pg.dense(0, n)
    want, av, mag = ref.attend(q[0].double(), K[0].nan_to_num(neginf=-1e30), V[0], (~gone)[None].expand(2, n), cfg.c().scale, 0.0)
    within(o[0], want, ref.attend_bound(want, av, mag, D, n, o.dtype, 0.0, 2.0 ** -17 if io == BF else 0.0), "some -inf")
    assert o[1].isnan().all() and o[2].isnan().all()
    check_attention(cfg, pg, q[3:], o[3:], 3, n - 1, 2.0 ** -17 if io == BF else 0.0, "clean")
    no_device_errors()


def test_decode_reports_bad_places():
    g = gen(4)
    cfg = lq.AttnConfig(4, 2, 64)
    pg = Paged(g, cfg, 3, 16, 2)
    pg.fill(g, [20, 20, 20])
    pg.table[1, 1] = 1 << 20
    q = randn(g, 3, 4, 64, dtype=torch.bfloat16)
    o = torch.full_like(q, 3.0)
    pos = torch.tensor([32, 19, 19], dtype=torch.int32, device="cuda")
    lq.lq_attn_decode(cfg, pg.cache, pos, q, o)
    assert lq.lq_device_errors() == lq.LQ_DEVERR_BAD_PAGE | lq.LQ_DEVERR_BAD_POSITION
    assert (o[0] == 3.0).all()
    check_attention(cfg, pg, q[2:], o[2:], 2, 19, 2.0 ** -17, "good sequence")


# ------------------------------------------------------------------ prefill

PREFILL_CASES = [
    # new tokens, starts, Hq, Hkv, D, page, window, softcap, io
    ([1], [0], 1, 1, 64, 16, 0, 0.0, BF),
    ([1, 1], [0, 200], 2, 1, 64, 16, 0, 0.0, F32),
    ([5, 0, 130, 64, 1], [0, 3, 7, 64, 15], 4, 2, 128, 16, 0, 0.0, BF),
    ([5, 0, 130, 64, 1], [0, 3, 7, 64, -1], 4, 2, 128, 16, 0, 0.0, F32),
    ([257, 129, 127], [0, 1, 300], 8, 1, 64, 32, 0, 0.0, BF),
    ([257, 129, 127], [0, 1, 300], 3, 3, 256, 64, 0, 0.0, BF),
    ([70, 33], [0, 1], 2, 1, 256, 64, 0, 25.0, F32),
    ([400, 300], [100, 0], 6, 2, 128, 64, 1, 0.0, BF),
    ([400, 300], [100, 0], 6, 2, 128, 256, 65, 30.0, BF),
    ([400, 300], [100, 0], 2, 2, 64, 128, 200, 10.0, F32),
    ([400, 300], [100, 0], 2, 1, 64, 128, 130, 10.0, BF),
    ([96, 96, 96, 96], [0, -1, 31, 500], 5, 5, 64, 32, 0, 0.0, BF),
    ([1000], [2111], 4, 1, 128, 64, 0, 0.0, BF),
]


@pytest.mark.parametrize("new,start,Hq,Hkv,D,page,window,softcap,io", PREFILL_CASES)
def test_prefill(new, start, Hq, Hkv, D, page, window, softcap, io):
    g = gen(Hq + D + len(new))
    dt = DT[io]
    cfg = lq.AttnConfig(Hq, Hkv, D, io_dtype=io, window=window, softcap=softcap)
    B = len(new)
    reach = [max(s, 0) + n for s, n in zip(start, new)]
    pg = Paged(g, cfg, B, page, -(-max(reach) // page))
    pg.fill(g, [r if s >= 0 else 0 for r, s in zip(reach, start)])
    uniform = len(set(new)) == 1
    T = sum(new) + (0 if uniform else 5)
    cu = None
    if not uniform:
        cu = torch.tensor([0] + torch.tensor(new).cumsum(0).tolist(), dtype=torch.int32, device="cuda")
    q = randn(g, T, Hq, D, dtype=dt, scale=2.0)
    o = torch.full((T, Hq, D), 3.0, dtype=dt, device="cuda")
    lq.lq_attn_prefill(cfg, pg.cache, torch.tensor(start, dtype=torch.int32, device="cuda"), cu, q, o)
    row = 0
    for b, (n, s) in enumerate(zip(new, start)):
        if n and s >= 0:
            check_attention(cfg, pg, q[row:row + n], o[row:row + n], b, s, 2.0 ** -8 if io == BF else 0.0, f"sequence {b}")
        else:
            assert (o[row:row + n] == 3.0).all()
        row += n
    assert (o[row:] == 3.0).all()
    no_device_errors()


# The same operator where calls are split differently: many rows (blocks of 32
# FP32 rows, several blocks to an SM), and few rows behind long contexts.
@pytest.mark.parametrize("new,start,Hq,Hkv,D,page,window,softcap,io", [
    ([700, 1, 500], [3, 200, 0], 24, 8, 128, 16, 0, 0.0, F32),
    ([640, 200], [0, 77], 32, 4, 64, 32, 150, 0.0, F32),
    ([300, 333], [40, 0], 16, 16, 256, 64, 0, 20.0, F32),
    ([900, 64, 1200], [100, 0, 7], 32, 4, 64, 32, 0, 0.0, BF),
    ([900, 64, 1200], [100, 0, 7], 16, 16, 64, 16, 333, 30.0, BF),
    ([2], [20000], 8, 2, 128, 64, 0, 0.0, BF),
    ([3, 1, 17], [5000, 9000, 250], 6, 2, 64, 16, 0, 0.0, BF),
    ([16, 16], [7000, 0], 4, 1, 256, 32, 0, 20.0, BF),
    ([5, 40], [9000, 600], 4, 4, 128, 16, 1000, 0.0, BF),
    ([5, 40], [9000, 600], 4, 4, 128, 16, 0, 0.0, F32),
    ([2], [20000], 8, 2, 64, 64, 0, 30.0, F32),
    ([1, 20, 3], [6000, 0, 100], 3, 1, 256, 128, 3000, 0.0, F32),
    ([4, 4, 4], [100, -1, 3000], 2, 2, 128, 16, 0, 0.0, F32),
])
def test_prefill_splits(new, start, Hq, Hkv, D, page, window, softcap, io):
    test_prefill(new, start, Hq, Hkv, D, page, window, softcap, io)


def test_prefill_reports_bad_places():
    g = gen(8)
    cfg = lq.AttnConfig(2, 1, 64)
    pg = Paged(g, cfg, 3, 16, 2)
    pg.fill(g, [32, 20, 20])
    pg.table[1, 0] = -3
    q = randn(g, 12, 2, 64, dtype=torch.bfloat16)
    o = torch.full_like(q, 3.0)
    # rows 2 and 3 of sequence 0 lie past its block table
    pos = torch.tensor([30, 16, 16], dtype=torch.int32, device="cuda")
    lq.lq_attn_prefill(cfg, pg.cache, pos, None, q, o)
    assert lq.lq_device_errors() == lq.LQ_DEVERR_BAD_PAGE | lq.LQ_DEVERR_BAD_POSITION
    assert (o[2:4] == 3.0).all()
    check_attention(cfg, pg, q[:2], o[:2], 0, 30, 2.0 ** -8, "rows inside the table")
    check_attention(cfg, pg, q[8:], o[8:], 2, 16, 2.0 ** -8, "good sequence")


# ------------------------------------------------------------------ streams, graphs, a run of them together

def test_decode_step_in_a_graph_and_on_another_stream():
    """append + decode captured once and replayed with other inputs, positions
    and pages equals the eager calls; another stream than the current one."""
    g = gen(21)
    cfg = lq.AttnConfig(8, 2, 128, norm=lq.LQ_NORM_RMS, rot_dim=64)
    B, page, width = 6, 16, 40
    pg = Paged(g, cfg, B, page, width)
    pg.fill(g, [width * page - 1] * B)
    w = 1 + 0.2 * randn(g, 128)
    cs = ref.table(64, width * page).cuda()
    qkv = randn(g, B, 12 * 128, dtype=torch.bfloat16)
    pos = torch.tensor([0, 100, -1, 638, 17, 333], dtype=torch.int32, device="cuda")
    qo, o = (torch.zeros(B, 8, 128, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    ws = torch.empty(lq.lq_attn_workspace_bytes(cfg, B), dtype=torch.uint8, device="cuda")

    def step(stream=None):
        q, k, v = (qkv[:, a * 128:b * 128].view(B, -1, 128) for a, b in ((0, 8), (8, 10), (10, 12)))
        lq.lq_kv_append(cfg, pg.cache, pos, None, q, k, v, w, w, cs, qo, stream=stream)
        lq.lq_attn_decode(cfg, pg.cache, pos, qo, o, ws, stream=stream)

    step()  # first calls set kernel attributes
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for i in range(3):
        qkv.copy_(randn(g, *qkv.shape, dtype=torch.bfloat16))
        pos.add_((pos >= 0).int() * (pos < 630).int())
        pg.table.copy_(pg.table.flip(0))
        o.zero_()
        graph.replay()
        got = o.clone()
        o.zero_()
        other = torch.cuda.Stream()
        other.wait_stream(torch.cuda.current_stream())
        step(stream=other)
        torch.cuda.current_stream().wait_stream(other)
        assert torch.equal(got, o)
        for b in range(B):
            if pos[b] >= 0:
                check_attention(cfg, pg, qo[b:b + 1], o[b:b + 1], b, int(pos[b]), 2.0 ** -17, f"step {i}, sequence {b}")
    no_device_errors()


@pytest.mark.parametrize("io", [BF, F32])
def test_prefill_then_decode_of_a_layer(io):
    """Prompts in two chunks, then single tokens: every output against the
    64-bit operators on the cache the calls built."""
    g = gen(31)
    dt = DT[io]
    Hq, Hkv, D, page = 6, 2, 64, 16
    cfg = lq.AttnConfig(Hq, Hkv, D, io_dtype=io, norm=lq.LQ_NORM_RMS, rot_dim=32, rot_pairs=lq.LQ_ROT_ADJACENT)
    B = 3
    pg = Paged(g, cfg, B, page, 20)
    w = 1 + 0.2 * randn(g, D)
    cs = ref.table(32, 320).cuda()
    pos = torch.zeros(B, dtype=torch.int32, device="cuda")
    prefill_split = 2.0 ** -8 if io == BF else 0.0
    for new in ([100, 7, 150], [33, 90, 1], [1, 1, 1], [1, 1, 1]):
        T = sum(new)
        n = torch.tensor(new, dtype=torch.int32, device="cuda")
        cu = torch.cat([n.new_zeros(1), n.cumsum(0).int()])
        qkv = randn(g, T, (Hq + 2 * Hkv) * D, dtype=dt)
        q, k, v = (qkv[:, a * D:b * D].view(T, -1, D) for a, b in ((0, 6), (6, 8), (8, 10)))
        qo, o = torch.empty(T, Hq, D, dtype=dt, device="cuda"), torch.empty(T, Hq, D, dtype=dt, device="cuda")
        one = T == B
        lq.lq_kv_append(cfg, pg.cache, pos, None if one else cu, q, k, v, w, w, cs, qo)
        if one:
            lq.lq_attn_decode(cfg, pg.cache, pos, qo, o)
        else:
            lq.lq_attn_prefill(cfg, pg.cache, pos, cu, qo, o)
        row = 0
        for b in range(B):
            check_attention(cfg, pg, qo[row:row + new[b]], o[row:row + new[b]], b, int(pos[b]),
                            (2.0 ** -17 if io == BF else 0.0) if one else prefill_split, f"{new} sequence {b}")
            row += new[b]
        pos += n
    no_device_errors()


def test_hybrid_step_feeds_the_linear_attention_decode():
    """L2-normalised q and k from the projection's slices into
    lq_decode_window: equal to the same call on rows normalised in 64 bits and
    rounded, where those agree bit for bit."""
    g = gen(41)
    B, H, d, W = 4, 3, 128, 8
    acfg = lq.AttnConfig(H, H, d, norm=lq.LQ_NORM_L2, eps=1e-6)
    cfg = lq.Config(batch=B, heads=H, window=W, n_comp=2)
    qk = randn(g, B, W, 2 * H * d, dtype=torch.bfloat16, scale=4.0)
    q, k = (qk[..., i * H * d:(i + 1) * H * d].unflatten(-1, (H, d)) for i in range(2))
    qn, kn = (torch.empty(B, W, H, d, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    lq.lq_qk_norm_rotate(acfg, q, k, None, None, None, None, qn, kn)
    v = randn(g, B, W, H, d, dtype=torch.bfloat16)
    alpha, beta = torch.rand(B, W, H, generator=g, device="cuda"), torch.rand(B, W, H, generator=g, device="cuda")
    outs = []
    for a, b in ((qn, kn), tuple(ref.norm_rotate(x, 1, 1e-6, None, 0, False, None, None)[0].to(torch.bfloat16) for x in (q, k))):
        st = lq.State(cfg)
        lq.lq_state_init(st)
        o = torch.empty(B, W, H, d, dtype=torch.bfloat16, device="cuda")
        lq.lq_decode_window(st, a.contiguous(), b.contiguous(), v, alpha, beta, W, o)
        outs.append(o.double())
    err = (outs[0] - outs[1]).norm() / outs[1].norm()
    # the two inputs differ by at most one BF16 step in the elements whose
    # quotient lies within FP32 rounding of a tie: far fewer than 1 in 1000
    assert err < 2.0 ** -8
    no_device_errors()


@pytest.mark.parametrize("Hq,Hkv,D,window,softcap,new,start", [
    (64, 1, 64, 0, 0.0, [4001, 130], [5, 0]),
    (64, 1, 64, 700, 20.0, [1500, 2600, 3], [0, 300, 64]),
    (32, 4, 128, 0, 0.0, [1900], [400]),
])
def test_prefill_of_many_rows(Hq, Hkv, D, window, softcap, new, start):
    """Long enough for blocks of the most rows (head size 64) and for several
    waves of blocks."""
    g = gen(Hq + D + window)
    cfg = lq.AttnConfig(Hq, Hkv, D, window=window, softcap=softcap)
    pg = Paged(g, cfg, len(new), 64, -(-max(n + s for n, s in zip(new, start)) // 64))
    pg.fill(g, [n + s for n, s in zip(new, start)])
    T = sum(new) + 2
    cu = torch.tensor([0] + torch.tensor(new).cumsum(0).tolist(), dtype=torch.int32, device="cuda")
    q = randn(g, T, Hq, D, dtype=torch.bfloat16, scale=2.0)
    o = torch.full((T, Hq, D), 3.0, dtype=torch.bfloat16, device="cuda")
    lq.lq_attn_prefill(cfg, pg.cache, torch.tensor(start, dtype=torch.int32, device="cuda"), cu, q, o)
    row = 0
    for b, (n, s) in enumerate(zip(new, start)):
        check_attention(cfg, pg, q[row:row + n], o[row:row + n], b, s, 2.0 ** -8, f"sequence {b}")
        row += n
    assert (o[row:] == 3.0).all()
    no_device_errors()


@pytest.mark.parametrize("io,split", [(BF, 2.0 ** -17), (F32, 0.0)])
@pytest.mark.parametrize("scale,softcap", [(0.3, 1e4), (0.3, 1.0), (-0.2, 10.0), (0.0, 0.0), (-0.1, 0.0), (3.0, 300.0)])
def test_scales_and_caps(io, split, scale, softcap):
    """Caps far above and well below the scores, scales of either sign and zero."""
    g = gen(int(1000 * scale) % 97 + int(softcap))
    cfg = lq.AttnConfig(4, 2, 64, io_dtype=io, scale=scale, softcap=softcap)
    n = 150
    pg = Paged(g, cfg, 2, 16, 10)
    pg.fill(g, [n, n])
    q = randn(g, 40, 4, 64, dtype=DT[io], scale=2.0)
    o = torch.empty_like(q)
    lq.lq_attn_prefill(cfg, pg.cache, torch.full((2,), n - 20, dtype=torch.int32, device="cuda"), None, q, o)
    for b in range(2):
        check_attention(cfg, pg, q[20 * b:20 * b + 20], o[20 * b:20 * b + 20], b, n - 20, 2.0 ** -8 if io == BF else 0.0, "prefill")
    qd, od = q[:2].contiguous(), torch.empty(2, 4, 64, dtype=DT[io], device="cuda")
    lq.lq_attn_decode(cfg, pg.cache, torch.full((2,), n - 1, dtype=torch.int32, device="cuda"), qd, od)
    for b in range(2):
        check_attention(cfg, pg, qd[b:b + 1], od[b:b + 1], b, n - 1, split, "decode")
    no_device_errors()


LONG_APPEND_CASES = [
    # as APPEND_CASES, over many blocks
    ([2000, 0, 1, 900, 700, 0, 1500], [0, 3, 60, -1, 7, 0, 1000], 16, 2, 256, 16, lq.LQ_NORM_RMS, 64, lq.LQ_ROT_HALVES, BF),
    ([800, 800, 800, 800], [5, -1, 0, 255], 32, 8, 128, 64, lq.LQ_NORM_L2, 128, lq.LQ_ROT_ADJACENT, BF),
    ([1300, 17, 2100], [100, 0, 31], 8, 4, 128, 32, lq.LQ_NORM_RMS, 48, lq.LQ_ROT_HALVES, F32),
    ([5000, 0, 4000], [0, 9, 300], 24, 8, 64, 256, lq.LQ_NORM_NONE, 0, 0, BF),
    ([1, 3000, 1], [8, 0, 8], 20, 5, 256, 128, lq.LQ_NORM_NONE, 256, lq.LQ_ROT_HALVES, F32),
]


@pytest.mark.parametrize("new,start,Hq,Hkv,D,page,norm,rot,pairs,io", LONG_APPEND_CASES)
@pytest.mark.parametrize("with_q", [True, False])
def test_long_append(new, start, Hq, Hkv, D, page, norm, rot, pairs, io, with_q):
    test_append(new, start, Hq, Hkv, D, page, norm, rot, pairs, io, with_q)


def test_long_norm_with_padding_positions_and_in_place():
    """Adjacent and split rotation over many tokens, q alone and in place."""
    for pairs, rot, io in ((lq.LQ_ROT_ADJACENT, 64, BF), (lq.LQ_ROT_HALVES, 128, F32)):
        test_norm_rotate(6001, 32, 8, 128, lq.LQ_NORM_RMS, True, rot, pairs, io)


def test_long_append_reports_bad_places():
    g = gen(10)
    cfg = lq.AttnConfig(32, 8, 128, rot_dim=128)
    B, n, page = 4, 1000, 64
    pg = Paged(g, cfg, B, page, 17)
    pg.table[1, 3] = pg.k.shape[0]   # tokens 192 .. 255 of sequence 1 have no page
    pg.table[2, 15] = -1             # tokens 960 .. of sequence 2
    k = randn(g, B * n, 8, 128, dtype=torch.bfloat16)
    q = randn(g, B * n, 32, 128, dtype=torch.bfloat16)
    qo = torch.full_like(q, 3.0)
    cs = ref.table(128, 1080).cuda()
    pos = torch.tensor([0, 0, 0, 100], dtype=torch.int32, device="cuda")  # the last 12 + 8 rows of sequence 3: past table and cache
    lq.lq_kv_append(cfg, pg.cache, pos, None, q, k, k, None, None, cs, qo)
    assert lq.lq_device_errors() == lq.LQ_DEVERR_BAD_PAGE | lq.LQ_DEVERR_BAD_POSITION
    gone = torch.zeros(B * n, dtype=torch.bool)
    gone[n + 192:n + 256] = True
    gone[2 * n + 960:3 * n] = True
    gone[3 * n + 980:] = True
    assert (qo[gone.cuda()] == 3.0).all() and (qo[~gone.cuda()] != 3.0).any(-1).any(-1).all()
    assert int((~pg.v.isnan()).sum()) == int((~gone).sum()) * 8 * 128


# ------------------------------------------------------------------ calls that share the GPU, far pages, odd scores

@pytest.mark.parametrize("io", [BF, F32])
def test_split_prefill_in_a_graph_and_on_another_stream(io):
    """Few rows behind long contexts, captured once and replayed with other
    positions (from a few keys to all), equal to the eager calls and right."""
    g = gen(51)
    cfg = lq.AttnConfig(8, 2, 128, io_dtype=io)
    B, n, page, width = 2, 3, 32, 200
    pg = Paged(g, cfg, B, page, width)
    pg.fill(g, [width * page] * B)
    q = randn(g, B * n, 8, 128, dtype=DT[io], scale=2.0)
    o = torch.zeros_like(q)
    pos = torch.tensor([0, 5000], dtype=torch.int32, device="cuda")
    lq.lq_attn_prefill(cfg, pg.cache, pos, None, q, o)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        lq.lq_attn_prefill(cfg, pg.cache, pos, None, q, o)
    for places in ([0, 5000], [6397, 255], [130, -1], [2047, 400]):
        pos.copy_(torch.tensor(places, dtype=torch.int32))
        o.fill_(3.0)
        graph.replay()
        got = o.clone()
        o.fill_(3.0)
        other = torch.cuda.Stream()
        other.wait_stream(torch.cuda.current_stream())
        lq.lq_attn_prefill(cfg, pg.cache, pos, None, q, o, stream=other)
        torch.cuda.current_stream().wait_stream(other)
        assert torch.equal(got, o)
        for b in range(B):
            if places[b] < 0:
                assert (o[b * n:(b + 1) * n] == 3.0).all()
            else:
                check_attention(cfg, pg, q[b * n:(b + 1) * n], o[b * n:(b + 1) * n], b, places[b],
                                2.0 ** -8 if io == BF else 0.0, f"{places} sequence {b}")
    no_device_errors()


def test_calls_on_two_streams_at_once():
    """Decode calls with workspaces of their own and split prefill calls, on two
    streams at once, give what they give alone."""
    g = gen(52)
    jobs = []
    for D, Hq, Hkv in ((128, 8, 2), (256, 4, 1)):
        cfg = lq.AttnConfig(Hq, Hkv, D)
        pg = Paged(g, cfg, 3, 64, 100)
        pg.fill(g, [6400] * 3)
        q = randn(g, 3, Hq, D, dtype=torch.bfloat16, scale=2.0)
        pos = torch.tensor([6399, 17, 3000], dtype=torch.int32, device="cuda")
        ws = torch.empty(lq.lq_attn_workspace_bytes(cfg, 3), dtype=torch.uint8, device="cuda")
        jobs.append((cfg, pg, pos, q, torch.empty_like(q), torch.empty_like(q), ws, torch.cuda.Stream()))

    def calls(job, stream):
        cfg, pg, pos, q, od, op, ws, _ = job
        lq.lq_attn_decode(cfg, pg.cache, pos, q, od, ws, stream=stream)
        lq.lq_attn_prefill(cfg, pg.cache, pos, None, q, op, stream=stream)

    alone = []
    for job in jobs:
        calls(job, None)
        alone.append((job[4].clone(), job[5].clone()))
        for b, p in enumerate((6399, 17, 3000)):
            check_attention(job[0], job[1], job[3][b:b + 1], job[4][b:b + 1], b, p, 2.0 ** -17, "decode")
            check_attention(job[0], job[1], job[3][b:b + 1], job[5][b:b + 1], b, p, 2.0 ** -8, "prefill")
    torch.cuda.synchronize()
    for _ in range(20):
        for job in jobs:
            calls(job, job[7])
    torch.cuda.synchronize()
    for job, (od, op) in zip(jobs, alone):
        assert torch.equal(job[4], od) and torch.equal(job[5], op)
    no_device_errors()


@pytest.mark.parametrize("io", [BF, F32])
def test_the_largest_batch(io):
    """4,096 sequences: decode, and prefill of one token each, idle slots among them."""
    g = gen(53)
    cfg = lq.AttnConfig(3, 1, 64, io_dtype=io, window=20)
    B = 4096
    pos = torch.randint(-1, 31, (B,), generator=g, device="cuda", dtype=torch.int32)
    pg = Paged(g, cfg, B, 16, 2)
    pl = pos.tolist()
    pg.fill(g, [p + 1 for p in pl])
    q = randn(g, B, 3, 64, dtype=DT[io], scale=2.0)
    od, op = torch.full_like(q, 3.0), torch.full_like(q, 3.0)
    lq.lq_attn_decode(cfg, pg.cache, pos, q, od)
    lq.lq_attn_prefill(cfg, pg.cache, pos, None, q, op)
    assert (od[pos < 0] == 3.0).all() and (op[pos < 0] == 3.0).all()
    for b in list(range(0, B, 97)) + [B - 1]:
        if pl[b] >= 0:
            check_attention(cfg, pg, q[b:b + 1], od[b:b + 1], b, pl[b], 2.0 ** -17 if io == BF else 0.0, f"decode {b}")
            check_attention(cfg, pg, q[b:b + 1], op[b:b + 1], b, pl[b], 2.0 ** -8 if io == BF else 0.0, f"prefill {b}")
    no_device_errors()


def test_pages_past_32_bits_of_elements():
    """A cache of more than 2^32 elements: append, decode and prefill at both of its ends."""
    g = gen(54)
    Hq, Hkv, D, page = 8, 4, 256, 256
    cfg = lq.AttnConfig(Hq, Hkv, D)
    P = (1 << 32) // (Hkv * D * page) + 40
    k = torch.empty(P, Hkv, page, D, dtype=torch.bfloat16, device="cuda")
    v = torch.empty_like(k)
    table = torch.tensor([[P - 1, 0, P - 2], [1, P - 30, 2]], dtype=torch.int32, device="cuda")
    cache = lq.KvCache(cfg, k, v, table)
    n = 700
    kk, vv = (randn(g, 2 * n, Hkv, D, dtype=torch.bfloat16) for _ in range(2))
    q = randn(g, 2 * n, Hq, D, dtype=torch.bfloat16, scale=2.0)
    qo, o = torch.empty_like(q), torch.empty_like(q)
    zero = torch.zeros(2, dtype=torch.int32, device="cuda")
    lq.lq_kv_append(cfg, cache, zero, None, q, kk, vv, None, None, None, qo)
    lq.lq_attn_prefill(cfg, cache, zero, None, qo, o)
    od = torch.empty(2, Hq, D, dtype=torch.bfloat16, device="cuda")
    lq.lq_attn_decode(cfg, cache, zero + n - 1, qo.view(2, n, Hq, D)[:, -1].contiguous(), od)
    assert torch.equal(qo, q)
    pos = torch.arange(n, device="cuda")[:, None]
    mask = torch.arange(n, device="cuda")[None] <= pos
    for b in range(2):
        rows = slice(b * n, (b + 1) * n)
        for x, y in ((k, kk), (v, vv)):
            got = x[table[b].long()].transpose(1, 2).reshape(-1, Hkv, D)[:n]
            assert torch.equal(got, y[rows])
        for h in range(Hq):
            K, V = (x[rows, h // 2].double() for x in (kk, vv))
            want, av, mag = ref.attend(q[rows, h].double(), K, V, mask, cfg.c().scale, 0.0)
            within(o[rows, h], want, ref.attend_bound(want, av, mag, D, n, o.dtype, 0.0, 2.0 ** -8), f"prefill {b} {h}")
            within(od[b, h], want[-1], ref.attend_bound(want[-1:], av[-1:], mag[-1:], D, n, o.dtype, 0.0, 2.0 ** -17)[0],
                   f"decode {b} {h}")
    no_device_errors()


@pytest.mark.parametrize("io,D", [(BF, 64), (BF, 128), (BF, 256), (F32, 64), (F32, 256)])
def test_prefill_infinite_scores(io, D):
    """-inf scores weigh nothing, also where they fill the keys of whole blocks
    of a split call; rows of nothing else are NaN, as their formula."""
    g = gen(55)
    cfg = lq.AttnConfig(2, 1, D, io_dtype=io)
    n, new = 4000, 2
    pg = Paged(g, cfg, 3, 16, -(-n // 16))
    pg.fill(g, [n] * 3)
    q = torch.zeros(3 * new, 2, D, dtype=DT[io], device="cuda")
    q[..., 0] = 1.0
    hit = torch.arange(n, device="cuda")
    gone = (hit < 2500) | (hit % 3 == 0)
    for b, t in ((0, hit[gone]), (1, hit)):
        pg.k[pg.table[b].long()[t // 16], 0, t % 16, 0] = -math.inf
    o = torch.empty_like(q)
    lq.lq_attn_prefill(cfg, pg.cache, torch.full((3,), n - new, dtype=torch.int32, device="cuda"), None, q, o)
    K, V = pg.dense(0, n)
    mask = (~gone)[None] & (hit[None] <= n - new + torch.arange(new, device="cuda")[:, None])
    for h in range(2):
        want, av, mag = ref.attend(q[:new, h].double(), K[0].nan_to_num(neginf=-1e30), V[0], mask, cfg.c().scale, 0.0)
        within(o[:new, h], want, ref.attend_bound(want, av, mag, D, n, o.dtype, 0.0, 2.0 ** -8 if io == BF else 0.0), "some -inf")
    assert o[new:2 * new].isnan().all()
    check_attention(cfg, pg, q[2 * new:], o[2 * new:], 2, n - new, 2.0 ** -8 if io == BF else 0.0, "clean")
    no_device_errors()


@pytest.mark.parametrize("T,Hq,Hkv,io", [(2000, 32, 8, BF), (900, 33, 11, F32), (3, 33, 11, BF), (1500, 40, 1, BF)])
def test_norm_rows_in_shares(T, Hq, Hkv, io):
    """Tokens whose heads take several blocks, in shares that do not divide them."""
    test_norm_rotate(T, Hq, Hkv, 256, lq.LQ_NORM_RMS, True, 64, lq.LQ_ROT_HALVES, io)
    test_norm_rotate(T, Hq, Hkv, 256, lq.LQ_NORM_L2, False, 256, lq.LQ_ROT_ADJACENT, io)


@pytest.mark.parametrize("new,start,Hq,Hkv,io", [([700, 1, 500], [3, 60, 0], 32, 8, BF), ([1, 2, 1], [0, 15, -1], 33, 11, F32)])
def test_append_rows_in_shares(new, start, Hq, Hkv, io):
    for with_q in (True, False):
        test_append(new, start, Hq, Hkv, 256, 32, lq.LQ_NORM_RMS, 64, lq.LQ_ROT_HALVES, io, with_q)
