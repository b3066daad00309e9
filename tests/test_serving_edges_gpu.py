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
