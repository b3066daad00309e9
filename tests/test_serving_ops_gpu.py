"""lt_attn_prompt, lt_attn_prefix and lt_verify_drafts against 64-bit forms, at
the sizes, layouts and masks where they can go wrong."""
import random

import pytest
import torch

import serving_ref as R

pytestmark = pytest.mark.gpu

DT = {"bf16": torch.bfloat16, "f32": torch.float32}


def _off(lens, dev="cuda"):
    o = [0]
    for n in lens:
        o.append(o[-1] + n)
    return torch.tensor(o, dtype=torch.int32, device=dev)


def _close(got, want, tol):
    bad = ~((got.double() - want).abs() <= tol)
    assert not bad.any(), (int(bad.sum()), got.double()[bad][:4].tolist(), want[bad][:4].tolist(),
                           tol[bad][:4].tolist())


# ---- attention over packed prompts -------------------------------------------------

def _prompt_inputs(dtype, H, Hk, hd, lq, lk, pad=0, fused=False, seed=0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    nq, nk = sum(lq) + pad, sum(lk) + pad
    if fused:
        x = torch.randn(nq, H + 2 * Hk, hd, generator=g, device="cuda").to(DT[dtype])
        return x[:, :H], x[:, H:H + Hk], x[:, H + Hk:]
    return tuple(torch.randn(n, h, hd, generator=g, device="cuda").to(DT[dtype])
                 for n, h in ((nq, H), (nk, Hk), (nk, Hk)))


PROMPTS = [
    # heads, kv heads, head_dim, query lengths, extra keys before each
    (16, 16, 128, [1], [0]),
    (4, 4, 32, [1, 1, 2, 1], [0, 0, 0, 0]),
    (4, 2, 128, [0, 5, 0, 0, 130, 0], [0] * 6),
    (2, 2, 64, [127, 128, 129, 255, 256, 257], [0] * 6),
    (55, 55, 96, [70], [0]),
    (8, 1, 128, [33, 200], [0, 0]),
    (6, 2, 64, [100, 43], [0, 11]),
    (14, 2, 96, [1, 90], [300, 7]),
    (64, 1, 32, [3, 17], [0, 1]),
    (4, 4, 128, [1, 1, 1], [1000, 63, 128]),
    (8, 2, 128, [64, 2, 600], [513, 1000, 1]),
    (4, 1, 128, [1300], [0]),
    (2, 1, 128, [700], [2000]),
]


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("H,Hk,hd,lq,ctx", PROMPTS)
def test_prompt_matches_64_bits(dtype, H, Hk, hd, lq, ctx):
    from looped_transformer_self_b200.binding import attn_prompt
    lk = [a + b if a else 0 for a, b in zip(lq, ctx)]
    q, k, v = _prompt_inputs(dtype, H, Hk, hd, lq, lk)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    got = attn_prompt(q, k, v, _off(lq), _off(lk), status=status)
    want, tol = R.prompt(q, k, v, lq, lk, hd ** -0.5)
    _close(got, want, tol)
    assert int(status) == 0


@pytest.mark.parametrize("group", [3, 5, 7, 11, 33, 48])
@pytest.mark.parametrize("hd", [32, 64, 96, 128])
def test_prompt_groups_that_do_not_fill_a_tile(group, hd):
    """Query heads per key/value head that do not divide 128: tiles of fewer rows."""
    from looped_transformer_self_b200.binding import attn_prompt
    lq, lk = [77, 1, 190], [77, 90, 400]
    q, k, v = _prompt_inputs("bf16", 2 * group, 2, hd, lq, lk)
    got = attn_prompt(q, k, v, _off(lq), _off(lk))
    want, tol = R.prompt(q, k, v, lq, lk, hd ** -0.5)
    _close(got, want, tol)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_prompt_fused_rows_padding_and_output_stride(dtype):
    """q, k, v as parts of one projection; rows behind the last sequence (NaN on
    input) stay as they were; the output is a part of a wider buffer."""
    from looped_transformer_self_b200.binding import attn_prompt
    H, Hk, hd, lq, pad = 8, 2, 64, [40, 1, 150], 9
    q, k, v = _prompt_inputs(dtype, H, Hk, hd, lq, lq, pad, fused=True)
    n = sum(lq)
    for t in (q, k, v):
        t[n:] = float("nan")
    buf = torch.full((n + pad, 2 * H, hd), 7.0, dtype=DT[dtype], device="cuda")
    got = attn_prompt(q, k, v, _off(lq), scale=0.3, out=buf[:, H:])
    want, tol = R.prompt(q[:n], k[:n], v[:n], lq, lq, 0.3)
    _close(got[:n], want, tol)
    assert bool((buf[n:] == 7).all()) and bool((buf[:, :H] == 7).all())


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_prompt_rows_without_keys_are_zero(dtype):
    """Fewer keys than queries: the first queries see nothing; a sequence with no keys at all."""
    from looped_transformer_self_b200.binding import attn_prompt
    lq, lk = [200, 7, 3], [50, 0, 3]
    q, k, v = _prompt_inputs(dtype, 4, 2, 64, lq, lk)
    got = attn_prompt(q, k, v, _off(lq), _off(lk))
    want, tol = R.prompt(q, k, v, lq, lk, 0.125)
    _close(got, want, tol)
    assert bool((got[:150] == 0).all()) and bool((got[200:207] == 0).all())


@pytest.mark.parametrize("bad", [float("nan"), float("inf"), float("-inf")])
@pytest.mark.parametrize("dtype,H,Hk,hd", [("bf16", 4, 2, 128), ("bf16", 2, 2, 96), ("f32", 4, 2, 64)])
def test_prompt_unseen_values_do_not_reach_a_row(dtype, H, Hk, hd, bad):
    """A bad key and value at token 150 of the middle sequence reach its rows from 150
    on and no other row: not the earlier ones, not the neighbours."""
    from looped_transformer_self_b200.binding import attn_prompt
    lq = [100, 300, 77]
    q, k, v = _prompt_inputs(dtype, H, Hk, hd, lq, lq)
    want, tol = R.prompt(q, k, v, lq, lq, hd ** -0.5)
    at = 250
    v[at, :, 5] = bad
    got = attn_prompt(q, k, v, _off(lq))
    fine = torch.ones(sum(lq), dtype=torch.bool, device="cuda")
    fine[at:400] = False
    _close(got[fine], want[fine], tol[fine])
    hit = got[at:400, :, 5].double()
    assert bool((hit.isnan() if bad != bad else (hit == bad)).all())
    other = [c for c in range(hd) if c != 5]
    _close(got[at:400][..., other], want[at:400][..., other], tol[at:400][..., other])
    k[at] = bad
    got = attn_prompt(q, k, v, _off(lq))
    _close(got[fine], want[fine], tol[fine])


def test_prompt_large_scores():
    """Scores in the thousands: the running maximum keeps the weights finite."""
    from looped_transformer_self_b200.binding import attn_prompt
    lq = [500]
    q, k, v = _prompt_inputs("bf16", 4, 4, 64, lq, lq)
    q *= 50
    k[250:] *= 30  # the maximum keeps rising
    got = attn_prompt(q, k, v, _off(lq))
    want, tol = R.prompt(q, k, v, lq, lq, 0.125)
    _close(got, want, tol)


def test_prompt_bad_offsets_are_reported_and_stay_in_range():
    from looped_transformer_self_b200.binding import attn_prompt
    q, k, v = _prompt_inputs("bf16", 4, 2, 64, [50], [50])
    for off in ([0, 80], [-5, 50], [40, 10], [0, 20, 10, 50]):
        status = torch.zeros(1, dtype=torch.int32, device="cuda")
        attn_prompt(q, k, v, torch.tensor(off, dtype=torch.int32, device="cuda"), status=status)
        assert int(status) == 4, off


# ---- attention of rows that share prefixes ------------------------------------------

def _prefix_inputs(dtype, H, Hk, hd, rows, np_, nt, slots=None, seed=0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    r = random.Random(seed)
    need = sum(np_) + sum(nt)
    slots = slots or need + 20
    cache = torch.randn(slots, 2, Hk * hd, generator=g, device="cuda").to(DT[dtype])
    order = list(range(slots))
    r.shuffle(order)
    prefixes, tails = [], []
    for n in np_:
        prefixes.append([order.pop() for _ in range(n)])
    for n in nt:
        tails.append([order.pop() for _ in range(n)])
    q = torch.randn(sum(rows), H, hd, generator=g, device="cuda").to(DT[dtype])
    return q, cache, prefixes, tails


def _lists(ll):
    return torch.tensor([x for l in ll for x in l], dtype=torch.int32, device="cuda"), _off([len(l) for l in ll])


def _prefix_call(q, cache, rows, prefixes, tails, **kw):
    from looped_transformer_self_b200.binding import attn_prefix
    p, po = _lists(prefixes)
    t, to = _lists(tails)
    return attn_prefix(q, cache, _off(rows), p, po, t, to, **kw)


PREFIXES = [
    # heads, kv heads, head_dim, rows of each group, prefix lengths, longest tail
    (16, 16, 128, [1], [1], 0),
    (16, 16, 128, [8], [601], 4),
    (4, 4, 32, [3, 1], [0, 70], 3),
    (55, 55, 96, [5], [130], 6),
    (8, 2, 128, [64], [1000], 33),
    (32, 8, 128, [7, 0, 20, 1], [500, 60, 64, 3], 150),
    (8, 1, 64, [40], [777], 9),
    (6, 2, 96, [30, 3], [65, 63], 5),
    (64, 1, 32, [3], [300], 2),
    (14, 2, 64, [19], [128], 64),
    (4, 1, 128, [2], [9000], 1),
    (2, 2, 128, [100], [256], 1),
]


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("H,Hk,hd,rows,np_,most", PREFIXES)
def test_prefix_matches_64_bits(dtype, H, Hk, hd, rows, np_, most):
    r = random.Random(sum(rows) + most)
    nt = [r.randint(0, most) for _ in range(sum(rows))]
    q, cache, prefixes, tails = _prefix_inputs(dtype, H, Hk, hd, rows, np_, nt)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    got = _prefix_call(q, cache, rows, prefixes, tails, status=status)
    want, tol = R.prefix(q, cache, rows, prefixes, tails, hd ** -0.5)
    _close(got, want, tol)
    assert int(status) == 0


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_prefix_padding_repeats_and_empty_rows(dtype):
    """Entries of -1 or past the cache are skipped, a slot may stand in several tails
    and twice in one; a row that sees nothing gets zeros; rows outside the groups stay."""
    from looped_transformer_self_b200.binding import attn_prefix
    rows, hd = [4, 3], 64
    q, cache, prefixes, tails = _prefix_inputs(dtype, 8, 2, hd, rows, [90, 0], [2] * 7)
    n = cache.shape[0]
    prefixes[0][5] = prefixes[0][80] = -1
    prefixes[0][17] = n
    tails[1] = [tails[0][0], tails[0][0], -1]
    tails[2] = []
    tails[4] = []
    tails[5] = [-1, n + 5, -7]
    extra = torch.randn(12, 8, hd, device="cuda").to(DT[dtype])
    extra[2:9] = q
    p, po = _lists(prefixes)
    t, to = _lists([[], []] + tails + [[], [], []])
    out = torch.full_like(extra, 3.0)
    ro = torch.tensor([2, 6, 9], dtype=torch.int32, device="cuda")
    attn_prefix(extra, cache, ro, p, po, t, to, out=out)
    want, tol = R.prefix(q, cache, rows, prefixes, tails, hd ** -0.5)
    _close(out[2:9], want, tol)
    assert bool((out[6:8] == 0).all()) and bool((out[:2] == 3).all()) and bool((out[9:] == 3).all())


@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
@pytest.mark.parametrize("dtype,H,Hk,hd", [("bf16", 8, 2, 128), ("bf16", 4, 4, 32), ("f32", 4, 2, 64)])
def test_prefix_unseen_values_do_not_reach_a_row(dtype, H, Hk, hd, bad):
    """A bad value in one row's tail reaches that row alone; bad slots that no list
    names reach nobody."""
    rows = [10]
    q, cache, prefixes, tails = _prefix_inputs(dtype, H, Hk, hd, rows, [100], [3] * 10)
    want, tol = R.prefix(q, cache, rows, prefixes, tails, hd ** -0.5)
    named = {s for l in prefixes + tails for s in l}
    for s in range(cache.shape[0]):
        if s not in named:
            cache[s] = bad
    kv = cache.view(-1, 2, Hk, hd)
    kv[tails[4][1], 1, :, 7] = bad
    got = _prefix_call(q, cache, rows, prefixes, tails)
    rest = [i for i in range(10) if i != 4]
    _close(got[rest], want[rest], tol[rest])
    hit = got[4, :, 7].double()
    assert bool((hit.isnan() if bad != bad else hit == bad).all())
    other = [c for c in range(hd) if c != 7]
    _close(got[4][:, other], want[4][:, other], tol[4][:, other])


# Sizes at which bf16 takes the tensor-core tiles (many keys): one short tile, tiles in both halves,
# ragged groups, several tiles per group, every head size, parts of odd lengths.
LONG_PREFIXES = [
    (16, 16, 128, [8], [10500], 4),
    (32, 8, 128, [32], [3100], 20),
    (32, 8, 128, [70, 1], [2500, 3000], 9),
    (8, 2, 64, [40, 0, 3, 9], [9000, 500, 700, 5000], 40),
    (55, 55, 96, [5, 2], [1500, 1601], 6),
    (14, 2, 96, [19], [13001], 64),
    (64, 1, 32, [3, 5], [24000, 300], 2),
    (6, 2, 128, [50], [12100], 0),
    (16, 16, 32, [1], [10127], 1),
    (16, 4, 128, [4] * 30, [260] * 30, 3),
]


@pytest.mark.parametrize("H,Hk,hd,rows,np_,most", LONG_PREFIXES)
def test_prefix_with_many_keys_matches_64_bits(H, Hk, hd, rows, np_, most):
    r = random.Random(sum(rows) + most)
    nt = [r.randint(0, most) for _ in range(sum(rows))]
    q, cache, prefixes, tails = _prefix_inputs("bf16", H, Hk, hd, rows, np_, nt)
    for p in prefixes:  # padding inside the lists
        for i in range(7, len(p), 991):
            p[i] = -1
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    out = torch.full_like(q, 3.0)
    got = _prefix_call(q, cache, rows, prefixes, tails, status=status, out=out)
    some = sorted(r.sample(range(sum(rows)), min(12, sum(rows))))
    first = [sum(rows[:g]) for g in range(len(rows))]
    for i in some:  # 64-bit rows one by one
        g = max(k for k in range(len(rows)) if first[k] <= i and rows[k])
        want, tol = R.prefix(q[i:i + 1], cache, [1], [prefixes[g]], [tails[i]], hd ** -0.5)
        _close(got[i:i + 1], want, tol)
    assert int(status) == 0
    again = _prefix_call(q, cache, rows, prefixes, tails)
    assert torch.equal(got, again)


@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
@pytest.mark.parametrize("H,Hk,hd,n", [(16, 16, 128, 10500), (32, 4, 96, 7000)])
def test_prefix_with_many_keys_keeps_unseen_values_out(H, Hk, hd, n, bad):
    """A bad value in one row's tail reaches that row alone, one in the prefix every row; bad
    slots that no list names reach nobody; a row without keys gets zeros."""
    rows = [9, 2]
    q, cache, prefixes, tails = _prefix_inputs("bf16", H, Hk, hd, rows, [n, 0], [3] * 11)
    tails[10] = [-1, -1]
    want, tol = R.prefix(q, cache, rows, prefixes, tails, hd ** -0.5)
    named = {s for l in prefixes + tails for s in l}
    rest = torch.tensor([s for s in range(cache.shape[0]) if s not in named], device="cuda")
    cache[rest] = bad
    kv = cache.view(-1, 2, Hk, hd)
    kv[tails[4][1], 1, :, 7] = bad
    got = _prefix_call(q, cache, rows, prefixes, tails)
    other = [c for c in range(hd) if c != 7]
    clean = [i for i in range(11) if i != 4]
    _close(got[clean], want[clean], tol[clean])
    _close(got[4][:, other], want[4][:, other], tol[4][:, other])
    hit = got[4, :, 7].double()
    assert bool((hit.isnan() if bad != bad else hit == bad).all()) and bool((got[10] == 0).all())
    kv[prefixes[0][n - 1], 1, :, 9] = bad  # the last key of the prefix: a block that holds tails too
    got = _prefix_call(q, cache, rows, prefixes, tails)
    hit = got[:9, :, 9].double()
    assert bool((hit.isnan() if bad != bad else hit == bad).all())
    _close(got[9:], want[9:], tol[9:])


def test_prefix_slots_past_two_gigabytes():
    """Cache offsets beyond 2^31 elements (and 2^32 bytes)."""
    H, hd, slots = 16, 128, 600_000
    cache = torch.zeros(slots, 2, H * hd, dtype=torch.bfloat16, device="cuda")
    g = torch.Generator(device="cuda").manual_seed(1)
    names = [slots - 1 - 7 * i for i in range(300)]
    cache[names] = torch.randn(300, 2, H * hd, generator=g, device="cuda").bfloat16()
    q = torch.randn(4, H, hd, generator=g, device="cuda").bfloat16()
    tails = [[names[290 + i]] for i in range(4)]
    got = _prefix_call(q, cache, [4], [names[:290]], tails)
    want, tol = R.prefix(q, cache, [4], [names[:290]], tails, hd ** -0.5)
    _close(got, want, tol)


def test_prefix_bad_offsets_are_reported_and_stay_in_range():
    from looped_transformer_self_b200.binding import attn_prefix
    q, cache, prefixes, tails = _prefix_inputs("bf16", 4, 2, 64, [6], [50], [2] * 6)
    p, po = _lists(prefixes)
    t, to = _lists(tails)
    good = dict(row_off=_off([6]), prefix_off=po, tail_off=to)
    i32 = lambda v: torch.tensor(v, dtype=torch.int32, device="cuda")  # noqa: E731
    for name, off in (("row_off", [0, 9]), ("row_off", [5, 2]), ("prefix_off", [0, 51]),
                      ("prefix_off", [-3, 50]), ("tail_off", [0, 2, 4, 3, 8, 10, 12]),
                      ("tail_off", [0, 2, 4, 6, 8, 10, 400])):
        a = dict(good, **{name: i32(off)})
        status = torch.zeros(1, dtype=torch.int32, device="cuda")
        attn_prefix(q, cache, a["row_off"], p, a["prefix_off"], t, a["tail_off"], status=status)
        assert int(status) == 4, (name, off)
    # groups that overlap make more tiles than the rows can have
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    n = 40
    over = i32([0, 6] * n + [0])
    attn_prefix(q, cache, over, p, i32([0] * (2 * n + 1)), t, to, status=status)
    assert int(status) == 4


# ---- verification ---------------------------------------------------------------------

def _verify_inputs(lens, V, seed, onehot=False, pad_cols=0):
    g = torch.Generator().manual_seed(seed)
    k, n = sum(lens), len(lens)
    z = torch.randn(k + n, V, generator=g) * 3
    p = torch.softmax(z, -1)
    if V > 8:
        p[p < 0.01 * p.amax(-1, keepdim=True)] = 0
        p = p / p.sum(-1, keepdim=True)
    trow = [i for s, m in enumerate(lens) for i in range(sum(lens[:s]) + s, sum(lens[:s]) + s + m)]
    q = torch.softmax(z[trow] + torch.randn(k, V, generator=g), -1)
    x = torch.multinomial(q, 1, generator=g)[:, 0] if k else torch.zeros(0, dtype=torch.long)
    ua, ud = torch.rand(k, generator=g), torch.rand(n, generator=g)
    return p, None if onehot else q, x.int(), ua, ud


def _verify_call(p, q, x, lens, ua, ud, **kw):
    from looped_transformer_self_b200.binding import verify_drafts
    acc, tok = verify_drafts(p.cuda(), None if q is None else q.cuda(), x.cuda(), _off(lens), ua.cuda(),
                             ud.cuda(), **kw)
    return acc.tolist(), tok.tolist()


@pytest.mark.parametrize("onehot", [False, True])
@pytest.mark.parametrize("V", [1, 2, 17, 500, 513, 4096, 49152, 65539])
@pytest.mark.parametrize("lens", [[0], [5], [3, 0, 1, 40, 2], [1] * 200])
def test_verify_matches_64_bits(lens, V, onehot):
    if V > 5000 and sum(lens) > 100:
        lens = lens[:20]
    p, q, x, ua, ud = _verify_inputs(lens, V, V + len(lens), onehot)
    got = _verify_call(p, q, x, lens, ua, ud)
    off = _off(lens, "cpu").tolist()
    assert got == R.verify(p, q, x.tolist(), off, ua, ud)


def test_verify_draws_at_the_ends_and_zero_mass():
    V = 1000
    p, q, x, ua, ud = _verify_inputs([2, 2, 2, 2, 1], V, 3)
    off = [0, 2, 4, 6, 8, 9]
    lens = [2, 2, 2, 2, 1]
    ua[:] = 0.999999
    ud[0], ud[1] = 0.0, 1 - 2.0 ** -24
    q[4] = p[6]                # residual without mass: drawn from p itself
    x[4] = int((p[6] == 0).nonzero()[0])
    p[9] = 0                   # a row without mass
    x[6] = -1                  # padding is not accepted
    x[8] = V                   # nor is a token past the vocabulary
    got = _verify_call(p, q, x, lens, ua, ud)
    assert got == R.verify(p, q, x.tolist(), off, ua, ud)
    p[0, 7], p[0, 9] = float("nan"), float("inf")
    p[2, :] = float("nan")
    got = _verify_call(p, q, x, lens, ua, ud)
    assert got == R.verify(p, q, x.tolist(), off, ua, ud)


def test_verify_strides_and_bad_offsets():
    from looped_transformer_self_b200.binding import verify_drafts
    lens, V = [3, 2], 1001
    p, q, x, ua, ud = _verify_inputs(lens, V, 5)
    want = R.verify(p, q, x.tolist(), [0, 3, 5], ua, ud)
    P = torch.full((7, V + 23), 9.0).cuda()
    P[:, :V] = p.cuda()
    Q = torch.full((5, V + 2), 9.0).cuda()
    Q[:, 1:V + 1] = q.cuda()
    acc, tok = verify_drafts(P[:, :V], Q[:, 1:V + 1], x.cuda(), _off(lens), ua.cuda(), ud.cuda())
    assert (acc.tolist(), tok.tolist()) == want
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    bad = torch.tensor([0, 3, 6], dtype=torch.int32, device="cuda")
    acc, tok = verify_drafts(P[:, :V], Q[:, 1:V + 1], x.cuda(), bad, ua.cuda(), ud.cuda(), status=status)
    assert acc.tolist() == [want[0][0], -1] and int(status) == 4


@pytest.mark.parametrize("onehot", [False, True])
@pytest.mark.parametrize("n,V", [(460, 33003), (200, 20000), (70, 4097)])
def test_verify_many_chains_with_infinities(n, V, onehot):
    """One, two and four CTAs a chain, several segments and groups a warp; entries that weigh nothing."""
    lens = [i % 2 for i in range(n)]
    p, q, x, ua, ud = _verify_inputs(lens, V, n, onehot)
    g = torch.Generator().manual_seed(n)
    for bad in (float("inf"), float("nan"), -float("inf")):
        rows = torch.arange(0, p.shape[0], 3)
        p[rows, torch.randint(V, rows.shape, generator=g)] = bad
        if q is not None:
            rows = torch.arange(0, q.shape[0], 2)
            q[rows, torch.randint(V, rows.shape, generator=g)] = bad
    ud[:4] = torch.tensor([0.0, 1 - 2.0 ** -24, 0.5, 1 - 2.0 ** -24])
    got = _verify_call(p, q, x, lens, ua, ud)
    assert got == R.verify(p, q, x.tolist(), _off(lens, "cpu").tolist(), ua, ud)


def test_verify_long_rows():
    """More segments than one round of a group's warps, and rows past 2^24 bytes."""
    V, lens = 9_000_001, [1, 0]
    g = torch.Generator().manual_seed(9)
    p = torch.rand(3, V, generator=g)
    p /= p.sum(-1, keepdim=True)
    x = torch.tensor([V - 5], dtype=torch.int32)
    for u in (0.0, 0.37, 0.83, 1 - 2.0 ** -24):
        ua, ud = torch.ones(1), torch.tensor([u, (u + 0.1) % 1])
        got = _verify_call(p, None, x, lens, ua, ud)
        assert got == R.verify(p, None, x.tolist(), [0, 1, 1], ua, ud)


# ---- together -----------------------------------------------------------------------

@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_prompt_cache_branches_and_verification_together(dtype):
    """A prompt goes through attn_prompt, its keys and values into cache slots; the next
    tokens' rows read them through attn_prefix.  Each branch equals attn_prompt over
    prompt + branch; a readout of the rows is verified."""
    from looped_transformer_self_b200.binding import attn_prompt, verify_drafts
    H, Hk, hd, n, m = 8, 2, 64, 333, 5
    q, k, v = _prompt_inputs(dtype, H, Hk, hd, [n + m], [n + m], seed=4)
    whole = attn_prompt(q, k, v, _off([n + m]))
    cache = torch.zeros(n + m + 50, 2, Hk * hd, dtype=DT[dtype], device="cuda")
    slots = torch.randperm(n + m + 50, generator=torch.Generator().manual_seed(2))[:n + m].tolist()
    cache[slots, 0], cache[slots, 1] = k.reshape(n + m, -1), v.reshape(n + m, -1)
    tails = [slots[n:n + i + 1] for i in range(m)]  # a chain: each row its ancestors and itself
    got = _prefix_call(q[n:], cache, [m], [slots[:n]], tails)
    want, tol = R.prompt(q, k, v, [n + m], [n + m], hd ** -0.5)
    _close(got, want[n:], tol[n:])
    _close(whole, want, tol)
    head = torch.randn(H * hd, 300, generator=torch.Generator(device="cuda").manual_seed(3), device="cuda")
    p = torch.softmax(got.float().reshape(m, -1) @ head, -1)
    d = torch.softmax(whole[n:n + m - 1].float().reshape(m - 1, -1) @ head, -1)
    x = d.argmax(-1).int()
    ua, ud = torch.rand(m - 1, device="cuda"), torch.rand(1, device="cuda")
    acc, tok = verify_drafts(p, d, x, _off([m - 1]), ua, ud)
    ref = R.verify(p.cpu(), d.cpu(), x.tolist(), [0, m - 1], ua.cpu(), ud.cpu())
    assert (acc.tolist(), tok.tolist()) == ref


def test_captured_graphs_follow_new_lengths_and_share_the_card():
    """The three calls captured once on a side stream; replays follow new offsets, and a
    second graph with its own scratch may replay beside the first."""
    from looped_transformer_self_b200 import binding as B
    H, Hk, hd, cap = 8, 2, 128, 400
    outs = []
    for which in range(2):
        q, k, v = _prompt_inputs("bf16", H, Hk, hd, [cap], [cap], seed=which)
        cache = torch.stack([k.reshape(cap, -1), v.reshape(cap, -1)], 1).contiguous()
        s = torch.cuda.Stream()
        qo = _off([cap])
        ro, po = _off([4]), _off([100])
        pre = torch.arange(cap, dtype=torch.int32, device="cuda")
        to = _off([1] * cap)
        p, dq, x, ua, ud = (t.cuda() for t in _verify_inputs([4], 2000, which))
        vo = _off([4])
        o1, o2 = torch.zeros_like(q), torch.zeros_like(q)
        sc1 = B.attn_prompt_scratch(q, k, qo)
        sc2 = B.attn_prefix_scratch(q, cache, ro)
        torch.cuda.synchronize()

        def step():
            B.attn_prompt(q, k, v, qo, out=o1, scratch=sc1)
            B.attn_prefix(q, cache, ro, pre, po, pre, to, out=o2, scratch=sc2)
            return B.verify_drafts(p, dq, x, vo, ua, ud)

        with torch.cuda.stream(s):
            step()
        s.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=s):
            res = step()
        # the graph reads every tensor of the calls, the offsets vo among them
        outs.append((g, s, q, k, v, cache, qo, ro, po, pre, to, o1, o2, res, (p, dq, x, ua, ud), (sc1, sc2, vo)))
    for lens, rows, np_ in (([cap], 4, 100), ([17, 300], 9, 399), ([1], 1, 0)):
        for g, s, q, k, v, cache, qo, ro, po, pre, to, o1, o2, res, ver, _ in outs:
            qo.copy_(torch.tensor([0, sum(lens)], dtype=torch.int32))
            ro.copy_(torch.tensor([0, rows], dtype=torch.int32))
            po.copy_(torch.tensor([0, np_], dtype=torch.int32))
            o1.zero_(), o2.zero_()
        torch.cuda.synchronize()
        for _ in range(3):
            for g, s, *_rest in outs:
                with torch.cuda.stream(s):
                    g.replay()
        torch.cuda.synchronize()
        for g, s, q, k, v, cache, qo, ro, po, pre, to, o1, o2, res, ver, _ in outs:
            n = sum(lens)
            want, tol = R.prompt(q[:n], k[:n], v[:n], [n], [n], hd ** -0.5)
            _close(o1[:n], want, tol)
            assert bool((o1[n:] == 0).all())
            want, tol = R.prefix(q[:rows], cache, [rows], [list(range(np_))], [[i] for i in range(rows)],
                                 hd ** -0.5)
            _close(o2[:rows], want, tol)
            assert bool((o2[rows:] == 0).all())
            p, dq, x, ua, ud = (t.cpu() for t in ver)
            assert (res[0].tolist(), res[1].tolist()) == R.verify(p, dq, x.tolist(), [0, 4], ua, ud)


def test_given_stream_and_repeatable_bits():
    from looped_transformer_self_b200 import binding as B
    q, k, v = _prompt_inputs("bf16", 8, 2, 64, [300, 100], [300, 100])
    a = B.attn_prompt(q, k, v, _off([300, 100]))
    rows, tails = [20], [[i] for i in range(20)]
    cache = torch.randn(900, 2, 128, device="cuda").bfloat16()
    b = _prefix_call(q[:20], cache, rows, [list(range(100, 900))], tails)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    a2 = B.attn_prompt(q, k, v, _off([300, 100]), stream=s)
    s.synchronize()
    b2 = _prefix_call(q[:20], cache, rows, [list(range(100, 900))], tails)
    assert torch.equal(a, a2) and torch.equal(b, b2)
