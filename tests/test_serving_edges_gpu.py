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
