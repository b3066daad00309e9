"""NaN queries and keys in lt_attn_prefix and lt_attn_prompt: a row that sees a NaN score is NaN, never a row
of zeros, and no other row is touched."""
import random

import pytest
import torch

import serving_ref as R

pytestmark = pytest.mark.gpu

DT = {"bf16": torch.bfloat16, "f32": torch.float32}
# fp32 tiles; bf16 tiles of 16, 32 and 64 rows; tensor-core tiles, with the rows in one and in both halves
SHAPES = [("f32", 4, 2, 64, [6, 2], [150, 90], 5), ("f32", 2, 2, 128, [70], [40], 3),
          ("bf16", 4, 4, 128, [6, 2], [150, 90], 5), ("bf16", 8, 2, 64, [6, 2], [301, 90], 5),
          ("bf16", 8, 2, 128, [12, 3], [301, 90], 5), ("bf16", 16, 2, 96, [12, 3], [200, 64], 70),
          ("bf16", 16, 16, 128, [6, 2], [10500, 200], 5), ("bf16", 32, 2, 64, [20, 3], [6300, 6301], 40)]


def _off(lens):
    o = [0]
    for n in lens:
        o.append(o[-1] + n)
    return torch.tensor(o, dtype=torch.int32, device="cuda")


def _flat(ll):
    return torch.tensor([x for l in ll for x in l], dtype=torch.int32, device="cuda")


def _case(dtype, H, Hk, hd, rows, np_, most):
    g = torch.Generator(device="cuda").manual_seed(sum(rows))
    r = random.Random(sum(rows))
    nt = [r.randint(1, most) for _ in range(sum(rows))]
    slots = sum(np_) + sum(nt)
    order = list(range(slots))
    r.shuffle(order)
    prefixes = [[order.pop() for _ in range(n)] for n in np_]
    tails = [[order.pop() for _ in range(n)] for n in nt]
    cache = torch.randn(slots, 2, Hk * hd, generator=g, device="cuda").to(DT[dtype])
    q = torch.randn(sum(rows), H, hd, generator=g, device="cuda").to(DT[dtype])
    return q, cache, prefixes, tails


def _call(q, cache, rows, prefixes, tails):
    from looped_transformer_self_b200.binding import attn_prefix
    return attn_prefix(q, cache, _off(rows), _flat(prefixes), _off([len(p) for p in prefixes]), _flat(tails),
                       _off([len(t) for t in tails]))


def _check(got, want, tol, nan):
    """Rows and heads marked in `nan` are NaN, the others as wanted."""
    assert bool(got[nan].isnan().all())
    bad = ~((got.double() - want).abs() <= tol)
    assert not bad[~nan].any()


@pytest.mark.parametrize("dtype,H,Hk,hd,rows,np_,most", SHAPES)
def test_prefix_nan_query(dtype, H, Hk, hd, rows, np_, most):
    q, cache, prefixes, tails = _case(dtype, H, Hk, hd, rows, np_, most)
    want, tol = R.prefix(q, cache, rows, prefixes, tails, hd ** -0.5)
    nan = torch.zeros(q.shape[:2], dtype=torch.bool, device="cuda")
    nan[1, 1] = nan[sum(rows) - 1, 0] = True
    q[1, 1, 3] = q[sum(rows) - 1, 0, hd - 1] = float("nan")
    _check(_call(q, cache, rows, prefixes, tails), want, tol, nan)


@pytest.mark.parametrize("dtype,H,Hk,hd,rows,np_,most", SHAPES)
def test_prefix_rows_that_see_only_nan_keys(dtype, H, Hk, hd, rows, np_, most):
    """The last group has no prefix; one of its rows sees only NaN keys, one only padding."""
    q, cache, prefixes, tails = _case(dtype, H, Hk, hd, rows, np_, most)
    rows, extra = rows + [3], [[tails[0][0], -1], [-1, -1], [prefixes[0][0]]]
    q = torch.cat([q, q[:3].flip(0)])
    cache = torch.cat([cache, cache[:1]])
    extra[0][0] = cache.shape[0] - 1  # a slot of its own
    prefixes, tails = prefixes + [[]], tails + extra
    want, tol = R.prefix(q, cache, rows, prefixes, tails, hd ** -0.5)
    cache[-1, 0, :] = float("nan")
    nan = torch.zeros(q.shape[:2], dtype=torch.bool, device="cuda")
    nan[sum(rows) - 3] = True
    got = _call(q, cache, rows, prefixes, tails)
    _check(got, want, tol, nan)
    assert bool((got[sum(rows) - 2] == 0).all())


@pytest.mark.parametrize("dtype,H,Hk,hd,rows,np_,most", SHAPES)
def test_prefix_one_nan_key_among_many(dtype, H, Hk, hd, rows, np_, most):
    """A NaN key of one head in one row's tail: that head's queries of that row; in a prefix: of the group."""
    q, cache, prefixes, tails = _case(dtype, H, Hk, hd, rows, np_, most)
    want, tol = R.prefix(q, cache, rows, prefixes, tails, hd ** -0.5)
    kv = cache.view(-1, 2, Hk, hd)
    share = H // Hk
    nan = torch.zeros(q.shape[:2], dtype=torch.bool, device="cuda")
    kv[tails[2][-1], 0, Hk - 1, 5] = float("nan")
    nan[2, (Hk - 1) * share:] = True
    _check(_call(q, cache, rows, prefixes, tails), want, tol, nan)
    kv[prefixes[0][-1], 0, 0, 7] = float("nan")
    nan[:rows[0], :share] = True
    _check(_call(q, cache, rows, prefixes, tails), want, tol, nan)


@pytest.mark.parametrize("dtype,H,Hk,hd", [("bf16", 4, 2, 128), ("bf16", 2, 2, 96), ("f32", 4, 2, 64)])
@pytest.mark.parametrize("lq,ctx", [([100, 300, 77], [0, 0, 0]), ([1, 9], [1500, 2000])])
def test_prompt_nan_query_and_keys(dtype, H, Hk, hd, lq, ctx):
    from looped_transformer_self_b200.binding import attn_prompt
    g = torch.Generator(device="cuda").manual_seed(7)
    lk = [a + b for a, b in zip(lq, ctx)]
    q = torch.randn(sum(lq), H, hd, generator=g, device="cuda").to(DT[dtype])
    k, v = (torch.randn(sum(lk), Hk, hd, generator=g, device="cuda").to(DT[dtype]) for _ in range(2))
    want, tol = R.prompt(q, k, v, lq, lk, hd ** -0.5)
    nan = torch.zeros(q.shape[:2], dtype=torch.bool, device="cuda")
    q[lq[0], 1, 0] = float("nan")
    nan[lq[0], 1] = True
    _check(attn_prompt(q, k, v, _off(lq), _off(lk)), want, tol, nan)
    k[0, Hk - 1, 0] = float("nan")  # seen by the whole first sequence
    nan[:lq[0], (Hk - 1) * (H // Hk):] = True
    _check(attn_prompt(q, k, v, _off(lq), _off(lk)), want, tol, nan)


@pytest.mark.parametrize("bad", [float("inf"), float("nan")])
@pytest.mark.parametrize("dtype,H,Hk,hd,rows,np_,most", SHAPES)
def test_prefix_bad_value_with_a_vanishing_weight(dtype, H, Hk, hd, rows, np_, most, bad):
    """A value that a row sees reaches it even where the weight is 0 in fp32: in its own tail, in the last
    block of the prefix, which holds tails too, and in a block without any."""
    q, cache, prefixes, tails = _case(dtype, H, Hk, hd, rows, np_, most)
    kv = cache.view(-1, 2, Hk, hd)
    q[:, :, 0] = 30.0
    kv[:, 0, :, 0] = 30.0
    seen = [tails[1][0], prefixes[0][-1], prefixes[0][0]]
    kv[seen, 0, :, 0] = -30.0  # scores 1800 / sqrt(hd) below the others
    want, tol = R.prefix(q, cache, rows, prefixes, tails, hd ** -0.5)
    hit = torch.zeros(q.shape, dtype=torch.bool, device="cuda")
    for i, s in enumerate(seen):
        kv[s, 1, :, 3 + i] = bad
        hit[1 if i == 0 else slice(0, rows[0]), :, 3 + i] = True
    got = _call(q, cache, rows, prefixes, tails)
    assert not bool(got[hit].isfinite().any())
    assert bool(((got.double() - want).abs() <= tol)[~hit].all())


@pytest.mark.parametrize("bad", [float("inf"), float("nan")])
@pytest.mark.parametrize("dtype,H,Hk,hd", [("bf16", 4, 2, 128), ("bf16", 2, 2, 96), ("f32", 4, 2, 64), ("f32", 1, 1, 32)])
def test_prompt_bad_value_with_a_vanishing_weight(dtype, H, Hk, hd, bad):
    from looped_transformer_self_b200.binding import attn_prompt
    g = torch.Generator(device="cuda").manual_seed(hd)
    n, at = 300, [5, 130, 270]
    q = torch.randn(n, H, hd, generator=g, device="cuda").to(DT[dtype])
    k, v = (torch.randn(n, Hk, hd, generator=g, device="cuda").to(DT[dtype]) for _ in range(2))
    q[:, :, 0] = 30.0
    k[:, :, 0] = 30.0
    k[at, :, 0] = -30.0
    want, tol = R.prompt(q, k, v, [n], [n], hd ** -0.5)
    hit = torch.zeros(n, H, hd, dtype=torch.bool, device="cuda")
    for i, s in enumerate(at):
        v[s, :, 3 + i] = bad
        hit[s:, :, 3 + i] = True
    got = attn_prompt(q, k, v, _off([n]))
    assert not bool(got[hit].isfinite().any())
    assert bool(((got.double() - want).abs() <= tol)[~hit].all())
