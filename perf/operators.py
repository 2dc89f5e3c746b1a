"""The softmax-attention operators of a hybrid linear-attention model as
measurable cases: per-head norm and rotation of q and k, the paged key-value
append, decode attention over the paged cache, and prefill attention.

``run`` computes a case in elementary torch operations (``own`` false) or
through the library's entry points (``own`` true) on the same inputs.
"""
from __future__ import annotations

import math
import random

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


# --------------------------------------------------------------------------
# Cases
# --------------------------------------------------------------------------

def listed():
    return [
        # one or two tokens of a decode step: launch latency is all there is
        dict(name="norm_step", op="norm", tokens=2, hq=32, hkv=8, d=128, norm="rms", rot=128,
             pairs="halves", dtype="bf16", mix=1),
        # q and k of a 2 x 8192 token prompt, L2-normalised for the linear-attention prefill
        dict(name="norm_l2_prompt", op="norm", tokens=16384, hq=32, hkv=32, d=128, norm="l2", rot=0,
             pairs="halves", dtype="bf16", mix=2),
        # an odd number of tokens, narrow heads, partial rotation of adjacent channels, FP32
        dict(name="norm_f32_odd", op="norm", tokens=1777, hq=12, hkv=4, d=64, norm="rms", rot=32,
             pairs="adjacent", dtype="f32", mix=3),
        # one decode step of a full batch: every sequence appends one token
        dict(name="append_step", op="append", batch=256, new_lo=1, new_hi=1, ctx_lo=0, ctx_hi=250,
             page=64, hq=32, hkv=8, d=128, norm="rms", rot=128, pairs="halves", dtype="bf16", mix=4),
        # prompts of uneven lengths enter the cache, wide heads, partial rotation
        dict(name="append_prompts", op="append", batch=13, new_lo=1, new_hi=1700, ctx_lo=0,
             ctx_hi=600, page=16, hq=16, hkv=2, d=256, norm="rms", rot=64, pairs="halves",
             dtype="bf16", mix=5),
        # the next token of a single short conversation: latency
        dict(name="decode_one", op="decode", batch=1, ctx_lo=700, ctx_hi=700, page=64, hq=32, hkv=8,
             d=128, window=0, softcap=0.0, dtype="bf16", mix=6),
        # a full decode batch with uneven contexts and a few idle slots
        dict(name="decode_batch", op="decode", batch=256, ctx_lo=15, ctx_hi=4095, page=64, hq=32,
             hkv=8, d=128, window=0, softcap=0.0, dtype="bf16", mix=7),
        # a few very long contexts: the split over the cache's length carries it
        dict(name="decode_long", op="decode", batch=3, ctx_lo=90000, ctx_hi=131071, page=16, hq=16,
             hkv=2, d=256, window=0, softcap=0.0, dtype="bf16", mix=8),
        # FP32 cache, capped scores, sliding window over uneven contexts
        dict(name="decode_f32_window", op="decode", batch=24, ctx_lo=1, ctx_hi=2999, page=32, hq=12,
             hkv=4, d=64, window=1000, softcap=30.0, dtype="f32", mix=9),
        # a 4096-token chunk of two long prompts on a cached prefix of the same length
        dict(name="prefill_chunk", op="prefill", batch=2, new_lo=4096, new_hi=4096, ctx_lo=4096,
             ctx_hi=4096, page=64, hq=32, hkv=8, d=128, window=0, softcap=0.0, dtype="bf16", mix=10),
        # prompts of uneven lengths in one call, sliding window and capped scores
        dict(name="prefill_ragged", op="prefill", batch=9, new_lo=1, new_hi=1500, ctx_lo=0,
             ctx_hi=900, page=32, hq=16, hkv=2, d=64, window=512, softcap=30.0, dtype="bf16", mix=11),
        # a short odd FP32 prompt per sequence
        dict(name="prefill_f32", op="prefill", batch=3, new_lo=200, new_hi=777, ctx_lo=0, ctx_hi=100,
             page=16, hq=8, hkv=8, d=128, window=0, softcap=0.0, dtype="f32", mix=12),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["norm", "append", "decode", "prefill"])
    dtype = rng.choice(["bf16", "bf16", "f32"])
    d = rng.choice([64, 128, 256])
    hkv = rng.choice([1, 2, 4, 5, 8])
    group = rng.choice([1, 2, 3, 4, 7, 8, 16])
    hq = hkv * group
    mix = rng.randrange(1 << 30)
    if op == "norm":
        rot = rng.choice([0, 16, d // 4, d // 2, d])
        tokens = max(1, min(_log_int(rng, 1, 16384), (1 << 26) // ((hq + hkv) * d)))
        return dict(op=op, tokens=tokens, hq=hq, hkv=hkv, d=d, norm=rng.choice(["l2", "rms"]), rot=rot,
                    pairs=rng.choice(["halves", "adjacent"]), dtype=dtype, mix=mix)
    page = rng.choice([16, 32, 64, 128])
    if op == "append":
        batch = _log_int(rng, 1, 256)
        new_hi = 1 if rng.random() < 0.4 else _log_int(rng, 2, 2000)
        new_hi = max(1, min(new_hi, (1 << 25) // ((hq + 2 * hkv) * d * batch)))
        return dict(op=op, batch=batch, new_lo=1, new_hi=new_hi, ctx_lo=0, ctx_hi=_log_int(rng, 1, 500),
                    page=page, hq=hq, hkv=hkv, d=d, norm=rng.choice(["none", "rms"]),
                    rot=rng.choice([0, 32, d // 2, d]), pairs=rng.choice(["halves", "adjacent"]),
                    dtype=dtype, mix=mix)
    window = rng.choice([0, 0, _log_int(rng, 1, 4000)])
    softcap = rng.choice([0.0, 0.0, 20.0, 50.0])
    if op == "decode":
        batch = _log_int(rng, 1, 256)
        most = (1 << 28) // (batch * hkv * d)
        ctx_hi = min(_log_int(rng, 1, 120000), most)
        return dict(op=op, batch=batch, ctx_lo=rng.choice([0, ctx_hi // 2, ctx_hi]), ctx_hi=ctx_hi,
                    page=page, hq=hq, hkv=hkv, d=d, window=window, softcap=softcap, dtype=dtype, mix=mix)
    batch = _log_int(rng, 1, 12)
    ctx_hi = rng.choice([0, _log_int(rng, 1, 2000)])
    new_hi = _log_int(rng, 2, 3000)
    most = (1 << 30) if dtype == "bf16" else (1 << 27)
    while new_hi > 2 and batch * hq * new_hi * (new_hi + ctx_hi) > most:
        new_hi = new_hi * 3 // 4
    return dict(op=op, batch=batch, new_lo=1, new_hi=new_hi, ctx_lo=0, ctx_hi=ctx_hi, page=page, hq=hq,
                hkv=hkv, d=d, window=window, softcap=softcap, dtype=dtype, mix=mix)


def _lengths(case):
    """(cached tokens, new tokens) of each sequence, by the case alone; a
    cached length of -1 is an idle slot."""
    r = random.Random(case["mix"])
    B = case["batch"]
    ctx = [r.randint(case["ctx_lo"], case["ctx_hi"]) for _ in range(B)]
    if case["op"] == "decode":
        new = [1] * B
    else:
        new = [r.randint(case["new_lo"], case["new_hi"]) for _ in range(B)]
    if B >= 16 and case["op"] in ("append", "decode"):
        for b in range(5, B, 37):
            ctx[b] = -1
    return ctx, new


def _norm_positions(case):
    """Positions of the norm case's tokens: far ones among them, -1 for padding."""
    r = random.Random(case["mix"])
    T = case["tokens"]
    start = r.randint(0, 30000)
    pos = [start + t for t in range(T)]
    if T >= 64:
        for t in range(11, T, 97):
            pos[t] = -1
    return pos


def _uniform(case):
    return case["op"] == "decode" or case["new_lo"] == case["new_hi"]


# --------------------------------------------------------------------------
# Inputs
# --------------------------------------------------------------------------

def _table(rot, length, dev):
    """cos, sin rows of the rotation angles pos * 1e6^(-2i/rot), in 64 bits, kept as FP32."""
    if rot == 0:
        return None
    inv = 1e6 ** (-torch.arange(0, rot, 2, dtype=torch.float64, device=dev) / rot)
    ang = torch.arange(length, dtype=torch.float64, device=dev)[:, None] * inv
    return torch.cat([ang.cos(), ang.sin()], 1).float()


def prepare(case, seed):
    dev = torch.device("cuda")
    gen = torch.Generator(device=dev)
    gen.manual_seed(seed)
    dt = DTYPES[case["dtype"]]
    hq, hkv, d = case["hq"], case["hkv"], case["d"]

    def randn(*shape, scale=1.0):
        return (torch.randn(*shape, generator=gen, device=dev) * scale).to(dt)

    def weight():
        return 1.0 + 0.2 * torch.randn(d, generator=gen, device=dev)

    st = {"case": dict(case)}
    if case["op"] == "norm":
        pos = _norm_positions(case)
        T = case["tokens"]
        # q and k as the two slices of one projection's output
        qk = randn(T, (hq + hkv) * d, scale=3.0)
        st.update(q=qk[:, :hq * d].view(T, hq, d), k=qk[:, hq * d:].view(T, hkv, d),
                  pos=torch.tensor(pos, dtype=torch.int32, device=dev),
                  table=_table(case["rot"], max(pos) + 1, dev),
                  q_out=torch.zeros(T, hq, d, dtype=dt, device=dev),
                  k_out=torch.zeros(T, hkv, d, dtype=dt, device=dev))
        st["wq"], st["wk"] = (weight(), weight()) if case["norm"] == "rms" else (None, None)
    else:
        ctx, new = _lengths(case)
        B, page = case["batch"], case["page"]
        need = [-(-(c + n) // page) if c >= 0 else 0 for c, n in zip(ctx, new)]
        width = max(max(need), 1)
        pages = sum(need) + 1  # one page is never handed out
        order = torch.randperm(pages - 1, generator=gen, device=dev).cpu().tolist()
        tab = torch.full((B, width), -1, dtype=torch.int32)
        at = 0
        for b in range(B):
            tab[b, :need[b]] = torch.tensor(order[at:at + need[b]], dtype=torch.int32)
            at += need[b]
        st["block_table"] = tab.to(dev)
        st["k_pages"] = randn(pages, hkv, page, d)
        st["v_pages"] = randn(pages, hkv, page, d)
        st["pos"] = torch.tensor(ctx, dtype=torch.int32, device=dev)
        cu = [0]
        for n in new:
            cu.append(cu[-1] + n)
        if _uniform(case):
            T = cu[-1]
            st["cu"] = None
        else:
            T = cu[-1] + 3  # rows behind the last sequence, as a padded batch has
            st["cu"] = torch.tensor(cu, dtype=torch.int32, device=dev)
        if case["op"] == "append":
            qkv = randn(T, (hq + 2 * hkv) * d, scale=3.0)
            st.update(q=qkv[:, :hq * d].view(T, hq, d),
                      k=qkv[:, hq * d:(hq + hkv) * d].view(T, hkv, d),
                      v=qkv[:, (hq + hkv) * d:].view(T, hkv, d),
                      table=_table(case["rot"], max(max(c + n for c, n in zip(ctx, new)), 1), dev),
                      q_out=torch.zeros(T, hq, d, dtype=dt, device=dev))
            st["wq"], st["wk"] = (weight(), weight()) if case["norm"] == "rms" else (None, None)
        else:
            # queries that pick out some keys: scores of a standard deviation of 2
            st["q"] = randn(T, hq, d, scale=2.0)
            st["o"] = torch.zeros(T, hq, d, dtype=dt, device=dev)
    if own:
        st.update(_handles(st))
    return st


def _handles(st):
    """What a user's program keeps between calls: the configuration, the cache
    object and the decode's workspace."""
    import linear_attention_recurrent_int8_b200 as lq
    c = st["case"]
    cfg = lq.AttnConfig(
        q_heads=c["hq"], kv_heads=c["hkv"], head_dim=c["d"],
        io_dtype=lq.LQ_BF16 if c["dtype"] == "bf16" else lq.LQ_F32,
        norm={"l2": lq.LQ_NORM_L2, "rms": lq.LQ_NORM_RMS}.get(c.get("norm"), lq.LQ_NORM_NONE),
        eps=1e-6, rot_dim=c.get("rot", 0),
        rot_pairs=lq.LQ_ROT_ADJACENT if c.get("pairs") == "adjacent" else lq.LQ_ROT_HALVES,
        scale=c["d"] ** -0.5, softcap=c.get("softcap", 0.0), window=c.get("window", 0))
    h = {"cfg": cfg}
    if "k_pages" in st:
        h["cache"] = lq.KvCache(cfg, st["k_pages"], st["v_pages"], st["block_table"])
    if c["op"] == "decode":
        h["ws"] = torch.empty(lq.lq_attn_workspace_bytes(cfg, c["batch"]), dtype=torch.uint8,
                              device="cuda")
    return h


# --------------------------------------------------------------------------
# The operators in elementary operations
# --------------------------------------------------------------------------

def _norm(x, kind, w):
    x = x.float()
    if kind == "l2":
        x = x * torch.rsqrt((x * x).sum(-1, keepdim=True) + 1e-6)
    elif kind == "rms":
        x = x * torch.rsqrt((x * x).mean(-1, keepdim=True) + 1e-6)
    return x if w is None else x * w


def _rotate(x, rot, pairs, table, pos):
    if rot == 0:
        return x
    row = table[pos.clamp(min=0).long()][:, None, :]
    c, s = row[..., :rot // 2], row[..., rot // 2:]
    if pairs == "halves":
        a, b = x[..., :rot // 2], x[..., rot // 2:rot]
        turned = torch.cat([a * c - b * s, b * c + a * s], -1)
    else:
        a, b = x[..., 0:rot:2], x[..., 1:rot:2]
        turned = torch.stack([a * c - b * s, b * c + a * s], -1).flatten(-2)
    return torch.cat([turned, x[..., rot:]], -1)


def _plain_norm(st):
    c, pos = st["case"], st["pos"]
    live = (pos >= 0)[:, None, None]
    for x, w, out in (("q", "wq", "q_out"), ("k", "wk", "k_out")):
        y = _rotate(_norm(st[x], c["norm"], st[w]), c["rot"], c["pairs"], st["table"], pos)
        st[out].copy_(torch.where(live, y.to(st[out].dtype), st[out]))
    return {"q": st["q_out"], "k": st["k_out"]}


def _token_places(st, T):
    """Sequence, position and liveness of each of the T token rows."""
    B = st["pos"].numel()
    t = torch.arange(T, device=st["pos"].device)
    if st["cu"] is None:
        n = T // B
        b, i = t // n, t % n
        live = st["pos"][b] >= 0
    else:
        cu = st["cu"].long()
        b = torch.searchsorted(cu, t, right=True) - 1
        live = b < B
        b = b.clamp(max=B - 1)
        i = t - cu[b]
        live = live & (st["pos"][b] >= 0)
    return b, i, st["pos"][b].long() + i, live


def _plain_append(st):
    c = st["case"]
    T, page = st["q"].shape[0], c["page"]
    b, _, pos, live = _token_places(st, T)
    spare = st["k_pages"].shape[0] - 1
    pid = st["block_table"][b, (pos.clamp(min=0) // page).clamp(max=st["block_table"].shape[1] - 1)]
    pid = torch.where(live, pid.long(), spare)
    off = torch.where(live, pos % page, 0)
    alive = live[:, None, None]
    q = _rotate(_norm(st["q"], c["norm"], st["wq"]), c["rot"], c["pairs"], st["table"], torch.where(live, pos, 0))
    k = _rotate(_norm(st["k"], c["norm"], st["wk"]), c["rot"], c["pairs"], st["table"], torch.where(live, pos, 0))
    for pages, new in ((st["k_pages"], k), (st["v_pages"], st["v"])):
        # a row that is not live writes back what the spare page holds
        val = torch.where(alive, new.to(pages.dtype), pages[spare, :, 0])
        pages.transpose(1, 2)[pid, off] = val
    st["q_out"].copy_(torch.where(alive, q.to(st["q_out"].dtype), st["q_out"]))
    return {"q": st["q_out"], "k_pages": st["k_pages"], "v_pages": st["v_pages"]}


def _dense(pages, table):
    """[B, hkv, tokens, d] in 32 bits of the pages in the table."""
    g = pages[table.long()].float()
    B, W, H, P, D = g.shape
    return g.permute(0, 2, 1, 3, 4).reshape(B, H, W * P, D)


def _plain_attention(st):
    c = st["case"]
    q, pos = st["q"], st["pos"]
    T, hq, d = q.shape
    B, hkv = pos.numel(), c["hkv"]
    n = 1 if c["op"] == "decode" else max(_lengths(c)[1])
    b, i, place, live = _token_places(st, T)
    if st["cu"] is None:
        rows = q.view(B, T // B, hq, d)
    else:
        at = (st["cu"][:-1].long()[:, None] + torch.arange(n, device=q.device)).clamp(max=T - 1)
        rows = q[at]
    rows = rows.float().view(B, n, hkv, hq // hkv, d).permute(0, 2, 3, 1, 4).reshape(B, hkv, -1, d)
    K, V = _dense(st["k_pages"], st["block_table"]), _dense(st["v_pages"], st["block_table"])
    s = torch.matmul(rows, K.transpose(-1, -2)).mul_(d ** -0.5)
    if c["softcap"] > 0:
        s = s.div_(c["softcap"]).tanh_().mul_(c["softcap"])
    s = s.view(B, hkv, hq // hkv, n, -1)
    key = torch.arange(s.shape[-1], device=q.device)
    mine = pos.clamp(min=0).long()[:, None, None] + torch.arange(n, device=q.device)[:, None]
    seen = key <= mine
    if c["window"] > 0:
        seen = seen & (key > mine - c["window"])
    s.masked_fill_(~seen[:, None, None], -math.inf)
    s = s.sub_(s.amax(-1, keepdim=True)).exp_()
    total = s.sum(-1, keepdim=True)
    y = torch.matmul(s.view(B, hkv, -1, s.shape[-1]), V).view(B, hkv, hq // hkv, n, d) / total
    y = y.permute(0, 3, 1, 2, 4).reshape(B, n, hq, d)[b, i.clamp(max=n - 1)]
    st["o"].copy_(torch.where(live[:, None, None], y.to(st["o"].dtype), st["o"]))
    return {"o": st["o"]}


# --------------------------------------------------------------------------
# The library's calls
# --------------------------------------------------------------------------

def _own(st):
    import linear_attention_recurrent_int8_b200 as lq
    op = st["case"]["op"]
    if op == "norm":
        lq.lq_qk_norm_rotate(st["cfg"], st["q"], st["k"], st["wq"], st["wk"], st["pos"], st["table"],
                             st["q_out"], st["k_out"])
        return {"q": st["q_out"], "k": st["k_out"]}
    if op == "append":
        lq.lq_kv_append(st["cfg"], st["cache"], st["pos"], st["cu"], st["q"], st["k"], st["v"], st["wq"],
                        st["wk"], st["table"], st["q_out"])
        return {"q": st["q_out"], "k_pages": st["k_pages"], "v_pages": st["v_pages"]}
    if op == "decode":
        lq.lq_attn_decode(st["cfg"], st["cache"], st["pos"], st["q"], st["o"], st["ws"])
        return {"o": st["o"]}
    lq.lq_attn_prefill(st["cfg"], st["cache"], st["pos"], st["cu"], st["q"], st["o"])
    return {"o": st["o"]}


def run(st):
    if own:
        return _own(st)
    op = st["case"]["op"]
    return _plain_norm(st) if op == "norm" else _plain_append(st) if op == "append" else _plain_attention(st)


# --------------------------------------------------------------------------
# What a pass cannot do without
# --------------------------------------------------------------------------

def _seen(p, window):
    """Keys that the query at position p attends to."""
    return min(p + 1, window) if window > 0 else p + 1


def work(case):
    es = 2 if case["dtype"] == "bf16" else 4
    hq, hkv, d = case["hq"], case["hkv"], case["d"]
    if case["op"] == "norm":
        live = sum(p >= 0 for p in _norm_positions(case))
        weights = 2 * 4 * d if case["norm"] == "rms" else 0
        return {"bytes": live * ((hq + hkv) * d * es * 2 + case["rot"] * 4 + 4) + weights,
                "flops": live * (hq + hkv) * (4 * d + 3 * case["rot"])}
    ctx, new = _lengths(case)
    if case["op"] == "append":
        live = sum(n for c, n in zip(ctx, new) if c >= 0)
        norm = 4 * d if case["norm"] == "rms" else 0
        return {"bytes": live * ((hq + 2 * hkv) * d * es * 2 + case["rot"] * 4),
                "flops": live * (hq + hkv) * (norm + 3 * case["rot"])}
    keys = pairs = rows = 0
    for c, n in zip(ctx, new):
        if c < 0:
            continue
        rows += n
        first = max(0, c + 1 - case["window"]) if case["window"] > 0 else 0
        keys += c + n - first
        pairs += sum(_seen(p, case["window"]) for p in range(c, c + n))
    return {"bytes": keys * hkv * d * 2 * es + rows * hq * d * 2 * es + -(-keys // case["page"]) * 4,
            "flops": pairs * hq * d * 4}


# --------------------------------------------------------------------------
# The definition in 64 bits
# --------------------------------------------------------------------------

def _exact_rows(x, w, table, pos, case):
    """Norm and rotation of rows x [T, H, d] at positions pos, channel pair by channel pair."""
    x = x.double()
    d, rot = case["d"], case["rot"]
    if case["norm"] != "none":
        m = x.square().sum(-1, keepdim=True)
        x = x / torch.sqrt((m if case["norm"] == "l2" else m / d) + 1e-6)
    if w is not None:
        x = x * w.double()
    y = x.clone()
    for i in range(rot // 2):
        a, b = (i, i + rot // 2) if case["pairs"] == "halves" else (2 * i, 2 * i + 1)
        z = torch.complex(table[pos, i].double(), table[pos, rot // 2 + i].double())[:, None]
        z = torch.complex(x[..., a], x[..., b]) * z
        y[..., a], y[..., b] = z.real, z.imag
    return y


def exact(case, seed):
    if own:
        raise RuntimeError("exact() is computed without the library")
    st = prepare(case, seed)
    if case["op"] == "norm":
        on = torch.tensor([t for t, p in enumerate(_norm_positions(case)) if p >= 0], device="cuda")
        out = {}
        for x, w in (("q", "wq"), ("k", "wk")):
            y = torch.zeros(st[x].shape, dtype=torch.float64, device="cuda")
            y[on] = _exact_rows(st[x][on], st[w], st["table"], st["pos"][on].long(), case)
            out[x] = y
        return out
    ctx, new = _lengths(case)
    page, d = case["page"], case["d"]
    if case["op"] == "append":
        q = torch.zeros(st["q"].shape, dtype=torch.float64, device="cuda")
        kp, vp = st["k_pages"].double(), st["v_pages"].double()
        row = 0
        for b, (c, n) in enumerate(zip(ctx, new)):
            if c >= 0:
                p = torch.arange(c, c + n, device="cuda")
                sl = slice(row, row + n)
                q[sl] = _exact_rows(st["q"][sl], st["wq"], st["table"], p, case)
                ids = st["block_table"][b].long()[p // page]
                kp[ids, :, p % page] = _exact_rows(st["k"][sl], st["wk"], st["table"], p, case)
                vp[ids, :, p % page] = st["v"][sl].double()
            row += n
        return {"q": q, "k_pages": kp, "v_pages": vp}
    o = torch.zeros(st["q"].shape, dtype=torch.float64, device="cuda")
    group = case["hq"] // case["hkv"]
    row = 0
    for b, (c, n) in enumerate(zip(ctx, new)):
        if c >= 0:
            ids = st["block_table"][b].long()[:-(-(c + n) // page)]
            p = torch.arange(c, c + n, device="cuda")[:, None]
            j = torch.arange(c + n, device="cuda")[None]
            hide = j > p
            if case["window"] > 0:
                hide = hide | (p - j >= case["window"])
            for h in range(case["hkv"]):
                K = st["k_pages"][ids, h].reshape(-1, d)[:c + n].double()
                V = st["v_pages"][ids, h].reshape(-1, d)[:c + n].double()
                Q = st["q"][row:row + n, h * group:(h + 1) * group].double()
                z = torch.einsum("tgd,jd->tgj", Q, K) / math.sqrt(d)
                if case["softcap"] > 0:
                    z = case["softcap"] * torch.tanh(z / case["softcap"])
                z = z.masked_fill(hide[:, None], -math.inf)
                a = torch.softmax(z, -1)
                o[row:row + n, h * group:(h + 1) * group] = torch.einsum("tgj,jd->tgd", a, V)
        row += n
    return {"o": o}
