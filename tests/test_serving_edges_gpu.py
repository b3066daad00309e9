"""lt_attn_prompt and lt_attn_prefix where counts are large: overlapping groups, many groups and sequences."""
import random

import pytest
import torch

import serving_ref as R

pytestmark = pytest.mark.gpu

DT = {"bf16": torch.bfloat16, "f32": torch.float32}


def _i32(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def _off(lens):
    o = [0]
    for n in lens:
        o.append(o[-1] + n)
    return _i32(o)


# dtype, rows, rows of a tile, keys: the fp32 tiles, the few-rows kernel (rows of 16) and the tensor-core
# tiles, each with few groups of several tiles and with so many that their units pass 32 bits
OVERLAPS = [("f32", 200, 64, 130, 3), ("bf16", 200, 16, 130, 20), ("bf16", 1000, 256, 200_000, 9),
            ("f32", 65535, 64, 300_000, 500), ("bf16", 65535, 16, 150_000, 5000), ("bf16", 65535, 256, 2_000_000, 600)]


@pytest.mark.parametrize("dtype,n_rows,tile,keys,times", OVERLAPS)
def test_overlapping_groups_are_reported_and_nothing_is_written(dtype, n_rows, tile, keys, times):
    """The same rows in every second group: more tiles than a call of so many rows and groups can have."""
    from looped_transformer_self_b200 import binding as B
    hd, groups = 32, 2 * times
    max_tiles = n_rows // tile + groups  # one key/value head
    blocks = keys // (128 if tile == 256 else 64)
    tiles = times * -(-n_rows // tile)
    if n_rows == 65535:
        assert tiles * blocks > 2 ** 31 > 2 * max_tiles * blocks
    q = torch.randn(n_rows, 1, hd, device="cuda").to(DT[dtype])
    cache = torch.randn(64, 2, hd, device="cuda").to(DT[dtype])
    ro = _i32([0, n_rows] * times + [n_rows])
    po = _i32([0, keys] * times + [keys])
    prefix = torch.arange(keys, dtype=torch.int32, device="cuda") % 64
    tail, to = _i32([]), torch.zeros(n_rows + 1, dtype=torch.int32, device="cuda")
    assert tiles > max_tiles
    out = torch.full_like(q, 3.0)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    scratch = B.attn_prefix_scratch(q, cache, ro).zero_()
    B.attn_prefix(q, cache, ro, prefix, po, tail, to, out=out, scratch=scratch, status=status)
    assert int(status) == 4 and bool((out == 3).all())


@pytest.mark.parametrize("dtype,keys", [("f32", 70), ("bf16", 70), ("bf16", 170_000)])
def test_overlapping_groups_that_fit_keep_the_other_rows(dtype, keys):
    """Overlaps within the scratch: reported, and the rows of the other groups are right."""
    from looped_transformer_self_b200 import binding as B
    g = torch.Generator(device="cuda").manual_seed(3)
    q = torch.randn(9, 1, 32, generator=g, device="cuda").to(DT[dtype])
    cache = torch.randn(keys, 2, 32, generator=g, device="cuda").to(DT[dtype])
    prefix = torch.arange(keys, dtype=torch.int32, device="cuda")
    ro, po = _i32([0, 5, 2, 5, 9]), _i32([0, 0, 0, 0, keys])
    to = torch.zeros(10, dtype=torch.int32, device="cuda")
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    got = B.attn_prefix(q, cache, ro, prefix, po, _i32([]), to, status=status)
    want, tol = R.attend(q[5:, 0], cache[:, 0], cache[:, 1], torch.ones(4, keys, dtype=torch.bool, device="cuda"),
                         32 ** -0.5)
    assert int(status) == 4
    assert bool(((got[5:, 0].double() - want).abs() <= tol).all())


@pytest.mark.parametrize("bad", [float("inf"), float("nan")])
@pytest.mark.parametrize("H,Hk,hd,rows,n,most", [(32, 4, 128, 30, 6000, 9), (64, 2, 96, 8, 14000, 60),
                                                 (8, 2, 64, 60, 12345, 20)])
def test_bad_tail_values_with_two_tiles_on_one_block(H, Hk, hd, rows, n, most, bad):
    """Both tiles of a call on the tensor-core tiles go over the same value rows; a bad value in each fourth
    row's tail reaches that row alone, run after run."""
    from looped_transformer_self_b200.binding import attn_prefix
    g = torch.Generator(device="cuda").manual_seed(rows)
    r = random.Random(rows)
    assert (H // Hk) * rows > 128
    nt = [r.randint(1, most) for _ in range(rows)]
    cache = torch.randn(n + sum(nt), 2, Hk * hd, generator=g, device="cuda").bfloat16()
    q = torch.randn(rows, H, hd, generator=g, device="cuda").bfloat16()
    order = list(range(n + sum(nt)))
    r.shuffle(order)
    tails = [[order.pop() for _ in range(m)] for m in nt]
    want, tol = R.prefix(q, cache, [rows], [order], tails, hd ** -0.5)
    hit = torch.zeros(rows, dtype=torch.bool, device="cuda")
    for i in range(0, rows, 4):
        cache[tails[i][-1], 1] = bad
        hit[i] = True
    args = (q, cache, _i32([0, rows]), _i32(order), _i32([0, n]), _i32([s for t in tails for s in t]), _off(nt))
    whole = None
    for _ in range(25):
        got = attn_prefix(*args)
        assert not bool(got[hit].isfinite().any())
        assert bool(((got[~hit].double() - want[~hit]).abs() <= tol[~hit]).all())
        bits = got.view(torch.int16)
        assert whole is None or torch.equal(bits, whole)
        whole = bits.clone()


@pytest.mark.parametrize("bad", [float("inf"), float("nan")])
def test_bad_values_of_the_last_block_with_two_tiles_on_it(bad):
    """A prompt whose two tiles end in the same block: a bad value at every fourth key of it."""
    from looped_transformer_self_b200.binding import attn_prompt
    H, Hk, hd, lq = 16, 2, 128, 30
    g = torch.Generator(device="cuda").manual_seed(2)
    q = torch.randn(lq, H, hd, generator=g, device="cuda").bfloat16()
    k, v = (torch.randn(lq, Hk, hd, generator=g, device="cuda").bfloat16() for _ in range(2))
    want, tol = R.prompt(q, k, v, [lq], [lq], hd ** -0.5)
    for i in range(14, lq, 4):
        v[i, :, i] = bad
    off, whole = _off([lq]), None
    reached = torch.zeros(lq, H, hd, dtype=torch.bool, device="cuda")
    for i in range(14, lq, 4):
        reached[i:, :, i] = True
    for _ in range(25):
        got = attn_prompt(q, k, v, off)
        assert not bool(got[reached].isfinite().any())
        assert bool(((got.double() - want).abs() <= tol)[~reached].all())
        bits = got.view(torch.int16)
        assert whole is None or torch.equal(bits, whole)
        whole = bits.clone()


@pytest.mark.parametrize("H,Hk,hd,lq,ctx", [(16, 16, 128, 256, 0), (55, 55, 96, 500, 0), (8, 2, 64, 640, 70),
                                            (4, 1, 128, 40, 3000), (6, 6, 32, 1000, 64)])
def test_infinities_in_blocks_that_one_tile_sees_whole(H, Hk, hd, lq, ctx):
    """Infinite values at keys that lie before all rows of a pair's second tile and among those of its first.
    Rows that do not see them are untouched; rows that do, however small their weight, are infinite, in every
    run alike."""
    from looped_transformer_self_b200.binding import attn_prompt
    g = torch.Generator(device="cuda").manual_seed(hd)
    lk = lq + ctx
    q = torch.randn(lq, H, hd, generator=g, device="cuda").bfloat16()
    k = torch.randn(lk, Hk, hd, generator=g, device="cuda").bfloat16()
    v = torch.randn(lk, Hk, hd, generator=g, device="cuda").bfloat16()
    want, tol = R.prompt(q, k, v, [lq], [lk], hd ** -0.5)
    tok = 128 // (H // Hk)
    at = ctx + tok // 2  # in the first tile's diagonal block
    first = at - ctx     # the first row that sees it
    v[at, :, 5] = float("inf")
    off, koff = _off([lq]), _off([lk])
    for far in (False, True):
        if far:  # a score far below the row's maximum: the weight is 0 in fp32
            q[:, :, 0] = 30.0
            k[:, :, 0] = 30.0
            k[at, :, 0] = -30.0
            want, tol = R.prompt(q, k, v.nan_to_num(posinf=0.0), [lq], [lk], hd ** -0.5)
        whole = None
        for _ in range(25):
            got = attn_prompt(q, k, v, off, koff)
            clean = got[:first].double()
            assert not bool(((clean - want[:first]).abs() > tol[:first]).any()) and bool(clean.isfinite().all())
            near = got[first:2 * tok, :, 5]  # rows of the pair: both tiles take the value out and give it back
            assert bool(near.isposinf().all())
            assert not bool(got[first:, :, 5].isfinite().any())
            rest = torch.cat([got[first:, :, :5], got[first:, :, 6:]], -1).double()
            other = torch.cat([want[first:, :, :5], want[first:, :, 6:]], -1)
            assert bool(((rest - other).abs() <= torch.cat([tol[first:, :, :5], tol[first:, :, 6:]], -1)).all())
            bits = got.view(torch.int16)
            assert whole is None or torch.equal(bits, whole)
            whole = bits.clone()


def _spot(q, cache, rows, prefixes, tails, got, n, r):
    """Some rows one by one against 64 bits."""
    first, hd = [sum(rows[:g]) for g in range(len(rows))], q.shape[2]
    for i in sorted(r.sample(range(sum(rows)), min(n, sum(rows)))):
        g = max(k for k in range(len(rows)) if first[k] <= i and rows[k])
        want, tol = R.prefix(q[i:i + 1], cache, [1], [prefixes[g]], [tails[i]], hd ** -0.5)
        assert bool(((got[i:i + 1].double() - want).abs() <= tol).all()), (i, g)


# groups: one row each (independent requests), rows of several tiles, empty groups in rows of their own
GROUPS = [([1] * 256, 40, 3), ([1] * 33, 700, 1), ([0] * 32 + [5, 0, 1] + [0] * 40 + [2], 300, 4),
          ([70, 0, 1] * 23, 90, 2), ([1] * 1000, 9, 2), ([3] * 64 + [0] * 64 + [200], 130, 5)]


@pytest.mark.parametrize("dtype,H,Hk,hd", [("bf16", 16, 16, 128), ("bf16", 8, 2, 64), ("bf16", 32, 2, 96),
                                           ("f32", 4, 2, 32)])
@pytest.mark.parametrize("rows,np_,most", GROUPS)
def test_more_groups_than_a_warp(dtype, H, Hk, hd, rows, np_, most):
    """More than 32 groups: the partition goes over them in steps."""
    from looped_transformer_self_b200.binding import attn_prefix
    r = random.Random(len(rows) + hd)
    g = torch.Generator(device="cuda").manual_seed(len(rows))
    lens = [r.randint(0, np_) for _ in rows]
    nt = [r.randint(1, most) for _ in range(sum(rows))]
    slots = 2 * max(np_, 2000)
    prefixes = [[r.randrange(-1, slots) for _ in range(n)] for n in lens]
    tails = [[r.randrange(slots) for _ in range(n)] for n in nt]
    cache = torch.randn(slots, 2, Hk * hd, generator=g, device="cuda").to(DT[dtype])
    q = torch.randn(sum(rows), H, hd, generator=g, device="cuda").to(DT[dtype])
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    args = (q, cache, _off(rows), _i32([s for p in prefixes for s in p]), _off(lens),
            _i32([s for t in tails for s in t]), _off(nt))
    got = attn_prefix(*args, status=status)
    assert int(status) == 0
    _spot(q, cache, rows, prefixes, tails, got, 25, r)
    assert torch.equal(got, attn_prefix(*args))


@pytest.mark.parametrize("dtype,H,Hk,hd", [("bf16", 16, 16, 128), ("bf16", 8, 2, 64), ("f32", 4, 2, 32)])
@pytest.mark.parametrize("n,most,ctx", [(33, 300, 0), (200, 40, 0), (100, 1, 500), (64, 260, 9), (500, 3, 2)])
def test_more_sequences_than_a_warp(dtype, H, Hk, hd, n, most, ctx):
    """More than 32 prompts, empty ones among them: a tile's sequence is found in steps."""
    from looped_transformer_self_b200.binding import attn_prompt
    r = random.Random(n + most)
    g = torch.Generator(device="cuda").manual_seed(n)
    lq = [r.randint(0, most) if i % 3 else most for i in range(n)]
    lk = [a + r.randint(0, ctx) if a else 0 for a in lq]
    q = torch.randn(sum(lq), H, hd, generator=g, device="cuda").to(DT[dtype])
    k, v = (torch.randn(sum(lk), Hk, hd, generator=g, device="cuda").to(DT[dtype]) for _ in range(2))
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    got = attn_prompt(q, k, v, _off(lq), _off(lk), status=status)
    assert int(status) == 0
    qo, ko = [sum(lq[:i]) for i in range(n)], [sum(lk[:i]) for i in range(n)]
    for i in r.sample([i for i in range(n) if lq[i]], 12) + [max(j for j in range(n) if lq[j])]:
        a, b = slice(qo[i], qo[i] + lq[i]), slice(ko[i], ko[i] + lk[i])
        want, tol = R.prompt(q[a], k[b], v[b], [lq[i]], [lk[i]], hd ** -0.5)
        assert bool(((got[a].double() - want).abs() <= tol).all()), i


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_prefix_on_a_decoders_own_plane(dtype):
    """The cache that a decode filled, plane by plane: the committed prefix's slots as the shared list, the
    last ones as the rows' own."""
    import synthetic as syn
    from looped_transformer_self_b200.binding import Decoder
    cfg = syn.MODELS["tiny"] if dtype == "f32" else syn.ModelConfig(
        "bf16_hd128", "bf16", 256, 2, 128, 512, 1000, 0, 3, 0, 4, resid_scale=0.5, head_gain=4.0, seed=7)
    dec = Decoder(cfg, syn.DecodeConfig(1, 2, 0.0, 1.0, 2, 32), syn.make_weights(cfg), max_branches=16, max_ctx=400)
    dec.prefill(syn.uniform_prompt(150, cfg.vocab, 1))
    dec.generate(20)
    slots = [x for x in dec.read_committed()[1][:-1] if x >= 0]
    assert len(slots) >= 150
    pool, p0 = dec.kv_pool()
    hd = cfg.d_model // cfg.n_heads
    g = torch.Generator(device="cuda").manual_seed(1)
    from looped_transformer_self_b200.binding import attn_prefix
    for plane in (p0, p0 + cfg.R - 1, p0 + cfg.n_core * cfg.R - 1):
        cache = pool[plane]
        q = torch.randn(3, cfg.n_heads, hd, generator=g, device="cuda").to(cache.dtype)
        prefix, tails = slots[:-3], [slots[-3:-2], slots[-3:-1], slots[-3:]]
        status = torch.zeros(1, dtype=torch.int32, device="cuda")
        got = attn_prefix(q, cache, _i32([0, 3]), _i32(prefix), _i32([0, len(prefix)]),
                          _i32([s for t in tails for s in t]), _off([1, 2, 3]), status=status)
        want, tol = R.prefix(q, cache, [3], [prefix], tails, hd ** -0.5)
        assert int(status) == 0 and bool(want.abs().amax() > 0)
        assert bool(((got.double() - want).abs() <= tol).all())
