"""What is measured of the serving operators: attention over packed prompts,
attention of rows that share a prefix, and the verification of drafted tokens.

A case names its operator in "op".  Lengths of ragged batches are drawn from
the case's own "mix" number, so they belong to the case; values come from the
seed that prepare() is given.
"""
import math
import random

import torch

own = False

# (query heads, key/value heads, head size): the heads of this repository's
# models (synthetic.MODELS: 4 x 32, 16 x 128, 55 x 96) and grouped ones.
HEADS = [(4, 4, 32), (16, 16, 128), (55, 55, 96), (32, 8, 128), (12, 4, 64), (8, 1, 128), (14, 2, 64)]
DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


# ---- cases ------------------------------------------------------------------

def listed():
    return [
        # one short prompt of the Ouro-1.4B heads: the prefill before a decode of the benchmark's kind
        dict(name="prompt_ouro_512", op="prompt", dtype="bf16", heads=16, kv_heads=16, head_dim=128,
             seqs=1, tokens=521, context=0, pad=0, fused=True, mix=1),
        # many users' prompts packed into one batch, from one token to over a thousand, grouped heads
        dict(name="prompt_packed_gqa", op="prompt", dtype="bf16", heads=32, kv_heads=8, head_dim=128,
             seqs=24, tokens=8192, context=0, pad=37, fused=True, mix=2),
        # one long document: the largest work
        dict(name="prompt_long_gqa", op="prompt", dtype="bf16", heads=32, kv_heads=8, head_dim=128,
             seqs=1, tokens=16384, context=0, pad=0, fused=False, mix=3),
        # a few new tokens on top of a long context each: a prompt taken in pieces
        dict(name="prompt_piece_context", op="prompt", dtype="bf16", heads=16, kv_heads=16, head_dim=128,
             seqs=2, tokens=150, context=6000, pad=0, fused=False, mix=4),
        # the Huginn-3.5B heads (55 x 96), two prompts
        dict(name="prompt_huginn", op="prompt", dtype="bf16", heads=55, kv_heads=55, head_dim=96,
             seqs=2, tokens=3001, context=0, pad=0, fused=True, mix=5),
        # the fp32 tiny model's prompts, single-token ones among them
        dict(name="prompt_tiny_f32", op="prompt", dtype="f32", heads=4, kv_heads=4, head_dim=32,
             seqs=9, tokens=700, context=0, pad=3, fused=True, mix=6),
        # a step's branches over a decode context of the benchmark's length (Ouro-1.4B)
        dict(name="prefix_ouro_600", op="prefix", dtype="bf16", heads=16, kv_heads=16, head_dim=128,
             groups=1, rows=8, prefix=601, tail=4, mix=7),
        # several prompts, some samples of each: ragged prefixes and group sizes, grouped heads
        dict(name="prefix_groups_gqa", op="prefix", dtype="bf16", heads=32, kv_heads=8, head_dim=128,
             groups=6, rows=40, prefix=4000, tail=150, mix=8),
        # a full branch table (64 rows) over a very long shared prefix
        dict(name="prefix_long_gqa", op="prefix", dtype="bf16", heads=32, kv_heads=8, head_dim=128,
             groups=1, rows=64, prefix=65431, tail=32, mix=9),
        # the fp32 tiny model's branches
        dict(name="prefix_tiny_f32", op="prefix", dtype="f32", heads=4, kv_heads=4, head_dim=32,
             groups=2, rows=11, prefix=777, tail=5, mix=10),
        # one request's drafts at the Ouro vocabulary: latency
        dict(name="verify_one", op="verify", seqs=1, drafts=5, vocab=49152, onehot=False, mix=11),
        # a batch of requests with ragged drafts (none for some) at the Huginn vocabulary
        dict(name="verify_batch", op="verify", seqs=192, drafts=6, vocab=65536, onehot=False, mix=12),
    ]


def _logint(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["prompt", "prompt", "prefix", "prefix", "verify"])
    mix = rng.randrange(1 << 30)
    if op == "verify":
        return dict(op=op, seqs=_logint(rng, 1, 192), drafts=rng.randrange(0, 13),
                    vocab=_logint(rng, 16, 100003), onehot=rng.random() < 0.4, mix=mix)
    dtype = "f32" if rng.random() < 0.25 else "bf16"
    h, hk, hd = rng.choice(HEADS)
    small = dtype == "f32"
    if op == "prompt":
        tokens = _logint(rng, 1, 2000 if small else 12000)
        context = _logint(rng, 1, 1000 if small else 8000) if rng.random() < 0.3 else 0
        if context:
            tokens = min(tokens, 2000)
        return dict(op=op, dtype=dtype, heads=h, kv_heads=hk, head_dim=hd,
                    seqs=_logint(rng, 1, min(tokens, 48)), tokens=tokens, context=context,
                    pad=rng.choice([0, 0, 1, 50]), fused=context == 0 and rng.random() < 0.5, mix=mix)
    groups = rng.choice([1, 1, 2, 5, 8])
    return dict(op=op, dtype=dtype, heads=h, kv_heads=hk, head_dim=hd, groups=groups,
                rows=_logint(rng, groups, 64),
                prefix=_logint(rng, 1, (3000 if small else 32768) // groups), tail=_logint(rng, 1, 200),
                mix=mix)


def _lengths(case):
    """The ragged lengths that the case stands for."""
    r = random.Random(case["mix"] * 7919 + 17)
    if case["op"] == "prompt":
        n, s = case["tokens"], case["seqs"]
        cuts = sorted(r.sample(range(1, n), s - 1)) if s > 1 else []
        q = [b - a for a, b in zip([0] + cuts, cuts + [n])]
        c = [r.randint(case["context"] // 2, case["context"]) for _ in q]
        return q, [a + b for a, b in zip(q, c)]
    if case["op"] == "prefix":
        g, m = case["groups"], case["rows"]
        cuts = sorted(r.sample(range(1, m), g - 1)) if g > 1 else []
        rows = [b - a for a, b in zip([0] + cuts, cuts + [m])]
        prefix = [case["prefix"]] + [r.randint(1, case["prefix"]) for _ in rows[1:]]
        tails = [r.randint(0 if p > 1 else 1, case["tail"]) for p, k in zip(prefix, rows) for _ in range(k)]
        return rows, prefix, tails
    return [r.randint(0, case["drafts"]) if i else case["drafts"] for i in range(case["seqs"])]


def _offsets(lens):
    off = [0]
    for n in lens:
        off.append(off[-1] + n)
    return off


def work(case):
    if case["op"] == "verify":
        s, rows = case["seqs"], 1 if case["onehot"] else 2
        k = sum(_lengths(case))
        # the row where a chain stops, two probabilities and two numbers a draft, the answers
        return {"bytes": s * rows * case["vocab"] * 4 + k * 16 + s * 16 + (k + s) * 4,
                "flops": s * case["vocab"] * 2}
    size = 4 if case["dtype"] == "f32" else 2
    h, hk, hd = case["heads"], case["kv_heads"], case["head_dim"]
    if case["op"] == "prompt":
        q, kv = _lengths(case)
        seen = sum(a * (b - a) + a * (a + 1) // 2 for a, b in zip(q, kv))
        return {"bytes": size * hd * (2 * h * sum(q) + 2 * hk * sum(kv)), "flops": 4 * hd * h * seen}
    rows, prefix, tails = _lengths(case)
    seen = sum(a * b for a, b in zip(rows, prefix)) + sum(tails)
    return {"bytes": size * hd * (2 * h * sum(rows) + 2 * hk * (sum(prefix) + sum(tails))),
            "flops": 4 * hd * h * seen}


# ---- inputs -----------------------------------------------------------------

def _ints(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    s = {"case": dict(case)}
    if case["op"] == "verify":
        lens = _lengths(case)
        k, n, V = sum(lens), len(lens), case["vocab"]
        off = _offsets(lens)
        # target rows: one a draft and one more a chain; draft rows follow the target's logits
        z = torch.randn(k + n, V, generator=g, device="cuda") * 3
        p = torch.softmax(z, -1)
        p = torch.where(p < 1e-2 * p.amax(-1, keepdim=True), torch.zeros_like(p), p)  # a truncated readout
        p = p / p.sum(-1, keepdim=True)
        trow = torch.tensor([off[i] + i + j for i in range(n) for j in range(lens[i])], dtype=torch.int64,
                            device="cuda")
        zq = z[trow] + torch.randn(k, V, generator=g, device="cuda")
        q = torch.softmax(zq, -1)
        noise = torch.rand(k, V, generator=g, device="cuda").clamp_min(1e-30).log().neg().log().neg()
        x = (zq + noise).argmax(-1) if k else torch.zeros(0, dtype=torch.int64, device="cuda")
        s.update(p=p, q=None if case["onehot"] else q, drafts=x.to(torch.int32), off=_ints(off), trow=trow,
                 lens=torch.tensor(lens, dtype=torch.int64, device="cuda"),
                 u_accept=torch.rand(k, generator=g, device="cuda"),
                 u_draw=torch.rand(n, generator=g, device="cuda"))
        return s
    dt = DTYPES[case["dtype"]]
    h, hk, hd = case["heads"], case["kv_heads"], case["head_dim"]
    if case["op"] == "prompt":
        lq, lkv = _lengths(case)
        nq, nkv = sum(lq) + case["pad"], sum(lkv) + case["pad"]
        if case["fused"]:  # the rows of one projection: a token's query heads, then its keys, then its values
            x = torch.randn(nq, h + 2 * hk, hd, generator=g, device="cuda").to(dt)
            q, k, v = x[:, :h], x[:, h:h + hk], x[:, h + hk:]
        else:
            q = torch.randn(nq, h, hd, generator=g, device="cuda").to(dt)
            k = torch.randn(nkv, hk, hd, generator=g, device="cuda").to(dt)
            v = torch.randn(nkv, hk, hd, generator=g, device="cuda").to(dt)
        s.update(q=q, k=k, v=v, lq=lq, lkv=lkv, q_off=_ints(_offsets(lq)), kv_off=_ints(_offsets(lkv)),
                 out=torch.zeros(nq, h, hd, dtype=dt, device="cuda"))
        return s
    rows, prefix, tails = _lengths(case)
    n = sum(prefix) + sum(tails)
    slots = n + 64
    cache = torch.randn(slots, 2, hk * hd, generator=g, device="cuda").to(dt)
    where = torch.arange(slots, device="cuda")
    # committed positions lie mostly in order, in runs that earlier pruning has moved about
    run = 16
    order = torch.randperm(-(-slots // run), generator=g, device="cuda")
    where = (order[:, None] * run + torch.arange(run, device="cuda")).reshape(-1)
    where = where[where < slots][:n].to(torch.int32)
    s.update(q=torch.randn(sum(rows), h, hd, generator=g, device="cuda").to(dt), cache=cache,
             prefix=where[:sum(prefix)].contiguous(), tail=where[sum(prefix):].contiguous(),
             rows=rows, prefix_lens=prefix, tails=tails, row_off=_ints(_offsets(rows)),
             prefix_off=_ints(_offsets(prefix)), tail_off=_ints(_offsets(tails)),
             out=torch.zeros(sum(rows), h, hd, dtype=dt, device="cuda"))
    return s


# ---- the operators ------------------------------------------------------------

def _run_own(s):
    from looped_transformer_self_b200 import binding as B
    op = s["case"]["op"]
    if op == "prompt":
        if "scratch" not in s:  # a program keeps its scratch memory
            s["scratch"] = B.attn_prompt_scratch(s["q"], s["k"], s["q_off"])
        return B.attn_prompt(s["q"], s["k"], s["v"], s["q_off"], s["kv_off"], out=s["out"],
                             scratch=s["scratch"])
    if op == "prefix":
        if "scratch" not in s:
            s["scratch"] = B.attn_prefix_scratch(s["q"], s["cache"], s["row_off"])
        return B.attn_prefix(s["q"], s["cache"], s["row_off"], s["prefix"], s["prefix_off"], s["tail"],
                             s["tail_off"], out=s["out"], scratch=s["scratch"])
    return B.verify_drafts(s["p"], s["q"], s["drafts"], s["off"], s["u_accept"], s["u_draw"])


def _plain_prompt(s):
    q, k, v, out = s["q"], s["k"], s["v"], torch.zeros_like(s["out"])
    h, hk, hd = q.shape[1], k.shape[1], q.shape[2]
    aq = ak = 0
    for lq, lk in zip(s["lq"], s["lkv"]):
        ks = k[ak:ak + lk].float().permute(1, 2, 0)  # [hk, hd, lk]
        vs = v[ak:ak + lk].float().transpose(0, 1)   # [hk, lk, hd]
        step = max(1, (1 << 28) // (h * lk))
        for a in range(0, lq, step):  # a piece of the rows whose scores fit the memory
            b = min(lq, a + step)
            see = lk - lq + b  # keys that the piece's last row sees
            qs = q[aq + a:aq + b].float().reshape(b - a, hk, h // hk, hd).permute(1, 2, 0, 3)
            z = torch.matmul(qs.reshape(hk, -1, hd), ks[:, :, :see]).view(h, b - a, see) * hd ** -0.5
            last = torch.arange(lk - lq + a, lk - lq + b, device=q.device)
            z.masked_fill_(torch.arange(see, device=q.device) > last[:, None], -math.inf)
            z = (z - z.amax(-1, keepdim=True)).exp_()
            o = torch.matmul(z.view(hk, -1, see), vs[:, :see]).view(h, b - a, hd) / z.sum(-1, keepdim=True)
            out[aq + a:aq + b] = o.transpose(0, 1).to(out.dtype)
        aq, ak = aq + lq, ak + lk
    return out


def _plain_prefix(s):
    q, cache, out = s["q"], s["cache"], torch.zeros_like(s["out"])
    h, hd = q.shape[1], q.shape[2]
    hk = cache.shape[2] // hd
    kv = cache.view(cache.shape[0], 2, hk, hd)
    own_off = s["tail_off"].long()
    r = p = 0
    for m, n in zip(s["rows"], s["prefix_lens"]):
        lens = own_off[r + 1:r + m + 1] - own_off[r:r + m]
        most = max(s["tails"][r:r + m])
        at = torch.arange(most, device=q.device)
        mine = at[None, :] < lens[:, None]  # [m, most]
        where = s["tail"].long()
        idx = (own_off[r:r + m, None] + at[None, :]).clamp(max=max(0, where.numel() - 1))
        tail = kv[where[idx]].float() if most else kv[:0].float().expand(m, 0, 2, hk, hd)
        shared = kv[s["prefix"][p:p + n].long()].float()  # [n, 2, hk, hd]
        qs = q[r:r + m].float().view(m, hk, h // hk, hd)
        z = torch.einsum("mkgd,nkd->mkgn", qs, shared[:, 0])
        zt = torch.einsum("mkgd,mtkd->mkgt", qs, tail[:, :, 0])
        zt = zt.masked_fill(~mine[:, None, None, :], -math.inf)
        w = torch.cat([z, zt], -1) * hd ** -0.5
        w = (w - w.amax(-1, keepdim=True)).exp()
        o = torch.einsum("mkgn,nkd->mkgd", w[..., :n], shared[:, 1])
        o = o + torch.einsum("mkgt,mtkd->mkgd", w[..., n:], tail[:, :, 1])
        out[r:r + m] = (o / w.sum(-1, keepdim=True)).reshape(m, h, hd).to(out.dtype)
        r, p = r + m, p + n
    return out


def _plain_verify(s):
    p, q, lens = s["p"], s["q"], s["lens"]
    n, k, V = lens.numel(), s["trow"].numel(), p.shape[1]
    off = s["off"][:-1].long()
    at = torch.arange(int(s["case"]["drafts"]) + 1, device=p.device)
    have = at[None, :] < lens[:, None]
    x = s["drafts"].long()
    idx = (off[:, None] + at[None, :]).clamp(max=max(0, k - 1))
    if k:
        px = p[s["trow"], x].double()
        qx = q[torch.arange(k, device=p.device), x].double() if q is not None else torch.ones_like(px)
        ok = (s["u_accept"].double() * qx < px)[idx] & have
    else:
        ok = have
    acc = ok.long().cumprod(1).sum(1)
    row = p[off + torch.arange(n, device=p.device) + acc].double()
    w = row.clone()
    if k:
        stop = (off + acc).clamp(max=k - 1)
        if q is not None:
            less = (p[off + torch.arange(n, device=p.device) + acc] - q[stop]).clamp_min(0).double()
        else:
            less = row.scatter(1, x[stop][:, None], 0.0)
        less = torch.where(less.sum(1, keepdim=True) > 0, less, row)
        w = torch.where((acc < lens)[:, None], less, row)
    c = w.cumsum(1)
    tok = (c > s["u_draw"].double()[:, None] * c[:, -1:]).long().argmax(1)
    out = torch.full((k + n,), -1, dtype=torch.int64, device=p.device)
    base = off + torch.arange(n, device=p.device)
    if k:
        put = at[None, :] < acc[:, None]
        out[(base[:, None] + at[None, :])[put]] = x[idx][put]
    out[base + acc] = tok
    return acc.to(torch.int32), out.to(torch.int32)


def run(state):
    if own:
        return _run_own(state)
    op = state["case"]["op"]
    if op == "prompt":
        return _plain_prompt(state)
    if op == "prefix":
        return _plain_prefix(state)
    return _plain_verify(state)


# ---- the definition in 64 bits --------------------------------------------------

def exact(case, seed):
    if case["op"] == "verify":
        return None  # whole numbers only
    s = prepare(case, seed)
    q = s["q"].double()
    h, hd = q.shape[1], q.shape[2]
    out = torch.zeros(q.shape, dtype=torch.float64, device=q.device)
    if case["op"] == "prompt":
        k, v = s["k"].double(), s["v"].double()
        share = h // k.shape[1]
        aq = ak = 0
        for lq, lk in zip(s["lq"], s["lkv"]):
            for i in range(h):
                for a in range(0, lq, 4096):
                    b = min(lq, a + 4096)
                    z = q[aq + a:aq + b, i] @ k[ak:ak + lk, i // share].T / math.sqrt(hd)
                    unseen = torch.ones(b - a, lk, dtype=torch.bool, device=q.device).triu(lk - lq + a + 1)
                    z[unseen] = -math.inf
                    w = torch.exp(z - torch.logsumexp(z, 1, keepdim=True))
                    out[aq + a:aq + b, i] = w @ v[ak:ak + lk, i // share]
            aq, ak = aq + lq, ak + lk
        return out
    hk = case["kv_heads"]
    r = p = t = 0
    for m, n in zip(s["rows"], s["prefix_lens"]):
        for i in range(r, r + m):
            seen = torch.cat([s["prefix"][p:p + n], s["tail"][t:t + s["tails"][i]]]).long()
            kv = s["cache"][seen].double().view(len(seen), 2, hk, hd).repeat_interleave(h // hk, 2)
            z = (kv[:, 0] * q[i]).sum(-1) / math.sqrt(hd)  # [seen, h]
            w = torch.exp(z - torch.logsumexp(z, 0))
            out[i] = (w[:, :, None] * kv[:, 1]).sum(0)
            t += s["tails"][i]
        r, p = r + m, p + n
    return out
