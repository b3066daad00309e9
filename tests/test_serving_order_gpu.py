"""One serving operator's output taken by the next with nothing between them: the
calls overlap on the device and still see each other's results.  Compared bit for
bit with the same calls and a synchronisation in between."""
import pytest
import torch

pytestmark = pytest.mark.gpu

DT = {"bf16": torch.bfloat16, "f32": torch.float32}
H, HD, N, ROWS, KEYS = 16, 128, 521, 8, 601  # a prompt of few items, a prefix call of few rows


def _i32(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def _inputs(dtype, seed, hd=HD):
    g = torch.Generator(device="cuda").manual_seed(seed)
    qkv = torch.randn(3, N, H, hd, generator=g, device="cuda").to(DT[dtype])
    cache = torch.randn(KEYS + ROWS, 2, H * hd, generator=g, device="cuda").to(DT[dtype])
    return qkv, cache


def _lists():
    return dict(row_off=_i32([0, ROWS]), prefix=torch.arange(KEYS, dtype=torch.int32, device="cuda"),
                prefix_off=_i32([0, KEYS]), tail=torch.arange(KEYS, KEYS + ROWS, dtype=torch.int32, device="cuda"),
                tail_off=torch.arange(ROWS + 1, dtype=torch.int32, device="cuda"))


@pytest.mark.parametrize("dtype,hd", [("bf16", 128), ("bf16", 96), ("bf16", 64), ("f32", 64)])
def test_prompt_output_is_the_next_calls_query(dtype, hd):
    from looped_transformer_self_b200.binding import attn_prefix, attn_prompt
    sets = [_inputs(dtype, s, hd) for s in range(3)]
    off, lists = _i32([0, N]), _lists()
    out = torch.zeros(N, H, hd, dtype=DT[dtype], device="cuda")
    wants = []
    for qkv, cache in sets:
        attn_prompt(*qkv, off, out=out)
        torch.cuda.synchronize()
        wants.append((out.clone(), attn_prefix(out[N - ROWS:], cache, **lists).clone()))
        torch.cuda.synchronize()
    got = []
    for i in range(60):
        qkv, cache = sets[i % 3]
        attn_prompt(*qkv, off, out=out)
        got.append((i, attn_prefix(out[N - ROWS:], cache, **lists)))
    torch.cuda.synchronize()
    for i, o in got:
        assert torch.equal(o, wants[i % 3][1]), i


@pytest.mark.parametrize("dtype,hd", [("bf16", 128), ("f32", 64)])
def test_prompt_output_is_the_next_calls_cache(dtype, hd):
    """The prompt writes into the cache rows that the prefix call reads."""
    from looped_transformer_self_b200.binding import attn_prefix, attn_prompt
    sets = [_inputs(dtype, s, hd) for s in range(3)]
    off, lists = _i32([0, N]), _lists()
    rows = [torch.randn(ROWS, H, hd, generator=torch.Generator(device="cuda").manual_seed(90 + s), device="cuda")
            .to(DT[dtype]) for s in range(3)]
    caches = [c.clone() for _, c in sets]
    wants = []
    for (qkv, _), cache, q in zip(sets, caches, rows):
        attn_prompt(*qkv, off, out=cache[:N, 1].unflatten(1, (H, hd)))
        torch.cuda.synchronize()
        wants.append(attn_prefix(q, cache, **lists).clone())
    shared = sets[0][1].clone()
    clean = torch.zeros_like(shared)
    for i in range(60):
        (qkv, first), q = sets[i % 3], rows[i % 3]
        clean.copy_(first)
        torch.cuda.synchronize()
        shared.copy_(clean)
        attn_prompt(*qkv, off, out=shared[:N, 1].unflatten(1, (H, hd)))
        got = attn_prefix(q, shared, **lists)
        assert torch.equal(got, wants[i % 3]), i


def test_memory_freed_between_the_calls():
    """A prompt's inputs freed behind its call go back to the stream's pool: the prefix call's output
    and scratch may take their place, and neither result changes."""
    from looped_transformer_self_b200.binding import attn_prefix, attn_prompt
    qkv, cache = _inputs("bf16", 5)
    off, lists = _i32([0, N]), _lists()
    q = torch.randn(ROWS, H, HD, generator=torch.Generator(device="cuda").manual_seed(6), device="cuda").bfloat16()
    want_a = attn_prompt(*qkv, off).clone()
    torch.cuda.synchronize()
    want_b = attn_prefix(q, cache, **lists).clone()
    torch.cuda.synchronize()
    for i in range(40):
        t = [x.clone() for x in qkv]
        a = attn_prompt(*t, off)
        del t
        b = attn_prefix(q, cache, **lists)
        assert torch.equal(a, want_a) and torch.equal(b, want_b), i


def test_prefix_output_overwritten_behind_it_and_verified_rows():
    """Three calls in a row, each on the last one's output; then the first one's inputs are overwritten."""
    from looped_transformer_self_b200.binding import attn_prefix, attn_prompt
    qkv, cache = _inputs("bf16", 8)
    off, lists = _i32([0, N]), _lists()
    keep = qkv.clone()
    out = torch.zeros(N, H, HD, dtype=torch.bfloat16, device="cuda")
    a = attn_prompt(*qkv, off, out=out)
    torch.cuda.synchronize()
    b = attn_prefix(a[:ROWS], cache, **lists)
    torch.cuda.synchronize()
    want = attn_prompt(b, qkv[1, :ROWS], qkv[2, :ROWS], _i32([0, ROWS])).clone()
    torch.cuda.synchronize()
    small = _i32([0, ROWS])
    for i in range(40):
        qkv.copy_(keep)
        attn_prompt(*qkv, off, out=out)
        b = attn_prefix(out[:ROWS], cache, **lists)
        c = attn_prompt(b, qkv[1, :ROWS], qkv[2, :ROWS], small)
        qkv.zero_()
        assert torch.equal(c, want), i


@pytest.mark.parametrize("dtype,hd", [("bf16", 128), ("f32", 64)])
def test_captured_chain_follows_new_inputs(dtype, hd):
    from looped_transformer_self_b200 import binding as B
    sets = [_inputs(dtype, s, hd) for s in range(3)]
    off, lists = _i32([0, N]), _lists()
    qkv, cache = sets[0][0].clone(), sets[0][1].clone()
    mid = torch.zeros(N, H, hd, dtype=DT[dtype], device="cuda")
    out = torch.zeros(ROWS, H, hd, dtype=DT[dtype], device="cuda")
    s1 = B.attn_prompt_scratch(qkv[0], qkv[1], off)
    s2 = B.attn_prefix_scratch(mid[:ROWS], cache, lists["row_off"])

    def step():
        B.attn_prompt(*qkv, off, out=mid, scratch=s1)
        B.attn_prefix(mid[N - ROWS:], cache, out=out, scratch=s2, **lists)

    wants = []
    for a, c in sets:
        qkv.copy_(a), cache.copy_(c)
        B.attn_prompt(*qkv, off, out=mid, scratch=s1)
        torch.cuda.synchronize()
        B.attn_prefix(mid[N - ROWS:], cache, out=out, scratch=s2, **lists)
        torch.cuda.synchronize()
        wants.append(out.clone())
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    side.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=side):
        for _ in range(3):  # a pass's prompt follows the last pass's merge without a wait on the host
            step()
    for i in range(20):
        with torch.cuda.stream(side):
            qkv.copy_(sets[i % 3][0]), cache.copy_(sets[i % 3][1])
            g.replay()
        side.synchronize()
        assert torch.equal(out, wants[i % 3]), i


def test_inputs_freed_behind_a_call_on_a_given_stream():
    """The given stream is busy when the call is made; its inputs are freed at once and their memory is asked
    for again on the current stream."""
    from looped_transformer_self_b200.binding import attn_prefix, attn_prompt, verify_drafts
    qkv, cache = _inputs("bf16", 11)
    lists, off = _lists(), _i32([0, N])
    g = torch.Generator(device="cuda").manual_seed(12)
    ver = [torch.rand(5, 4000, generator=g, device="cuda"), torch.rand(4, 4000, generator=g, device="cuda"),
           torch.randint(4000, (4,), generator=g, device="cuda", dtype=torch.int32), _i32([0, 4]),
           torch.rand(4, generator=g, device="cuda"), torch.rand(1, generator=g, device="cuda")]
    torch.cuda.synchronize()
    want = [attn_prompt(*qkv, off), attn_prefix(qkv[0, :ROWS], cache, **lists), *verify_drafts(*ver)]
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    for _ in range(5):
        t = [x.clone() for x in qkv] + [off.clone()]
        c, ls, vs = cache.clone(), {k: x.clone() for k, x in lists.items()}, [x.clone() for x in ver]
        torch.cuda.synchronize()
        with torch.cuda.stream(side):
            torch.cuda._sleep(20_000_000)  # about 10 ms
        got = [attn_prompt(*t, stream=side), attn_prefix(t[0][:ROWS], c, **ls, stream=side),
               *verify_drafts(*vs, stream=side)]
        sizes = [x.shape for x in [*t, c, *ls.values(), *vs]], [x.dtype for x in [*t, c, *ls.values(), *vs]]
        del t, c, ls, vs
        reused = [torch.zeros(s, dtype=d, device="cuda") for s, d in zip(*sizes)]
        side.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, want))
        del reused
