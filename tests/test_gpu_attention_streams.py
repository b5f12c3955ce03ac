"""Plans of rotary positions and attention called on another stream than the current one, or than the one they were
made on: the workspace is zeroed first, no output takes memory that is still read, inputs and plans may be dropped at
once, lens moves on only behind the step.  Each test holds one of the two streams back for some milliseconds."""
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

HOLD = 30_000_000                                    # clock cycles: some 15 ms
HEADS, KV, HD, N = 8, 2, 64, 600


def _rows(n, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return [torch.randn((n, w * HD), generator=g, device="cuda").bfloat16() for w in (HEADS, KV, KV, HEADS)]


def _decoder(lens, tokens=1):
    from dynamic_short_convolutions_b200 import ops

    dec = ops.AttnDecoder(torch.bfloat16, 2, HEADS, KV, HD, 4000, tokens, rope_table=ops.rope_table(4000, HD))
    g = torch.Generator(device="cuda").manual_seed(7)
    for c in (dec.k_cache, dec.v_cache):
        c.copy_(torch.randn(c.shape, generator=g, device="cuda"))
    dec.lens.fill_(lens)
    return dec


def _plans():
    """{name: (make, call(plan, stream) -> outputs)}"""
    from dynamic_short_convolutions_b200 import ops

    q, k, v, do = _rows(N, 1)
    cu = torch.tensor([0, 100, 350, 600], dtype=torch.int32, device="cuda")
    table = ops.rope_table(N, HD)
    attn = lambda: ops.AttnPlan(torch.bfloat16, 1, N, HEADS, KV, HD)

    def train(plan, s):
        o, lse = plan.forward(q, k, v, cu, want_lse=True, stream=s)
        return [o, lse, *plan.backward(do, q, k, v, o, lse, cu, stream=s).values()]

    return {"rope": (lambda: ops.RopePlan(torch.bfloat16, 1, N, HEADS, HD, table), lambda p, s: [p.apply(q, stream=s)]),
            "attention": (attn, train),
            "step": (lambda: _decoder(3500), lambda p, s: [p.step(q[:2], k[:2], v[:2], stream=s)]),
            "drafts": (lambda: _decoder(3500, 24), lambda p, s: [p.step(q[:48], k[:48], v[:48], stream=s)])}


@pytest.mark.parametrize("how", ["stream", "handle", "current"])
@pytest.mark.parametrize("name", ["rope", "attention", "step", "drafts"])
def test_a_plan_made_just_before(name, how):
    make, call = _plans()[name]
    want = call(make(), None)
    torch.cuda.synchronize()
    for t in vars(make()).values():                  # a block of garbage where the next workspace will lie
        if isinstance(t, torch.Tensor) and t.dtype == torch.uint8:
            t.fill_(255)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    torch.cuda._sleep(HOLD)
    plan = make()                                    # zeroed behind the hold
    if how == "current":
        with torch.cuda.stream(side):
            got = call(plan, None) if name in ("rope", "attention") else None
        if got is None:                              # its caches were filled here, which is the caller's to order
            side.wait_stream(torch.cuda.current_stream())
            with torch.cuda.stream(side):
                got = call(plan, None)
    else:
        got = call(plan, side if how == "stream" else side.cuda_stream)
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))


@pytest.mark.parametrize("name", ["rope", "attention", "step"])
def test_outputs_leave_memory_alone_that_is_still_read(name):
    make, call = _plans()[name]
    plan = make()
    want = call(plan, None)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    held = [torch.ones_like(t) for t in want]        # of the outputs' sizes, read behind the hold, dropped before it
    sums = [torch.zeros((), dtype=torch.float64, device="cuda") for _ in want]
    total = [t.numel() for t in want]
    torch.cuda.synchronize()
    torch.cuda._sleep(HOLD)
    for t, s in zip(held, sums):
        s.add_(t.double().sum())
    del held, t
    got = call(plan, side)
    torch.cuda.synchronize()
    assert [int(s) for s in sums] == total
    assert all(torch.equal(a, b) for a, b in zip(got, want))


@pytest.mark.parametrize("name", ["rope", "attention", "step", "drafts"])
def test_inputs_and_plans_dropped_at_once(name):
    make, call = _plans()[name]
    want = call(make(), None)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    make, call = _plans()[name]
    with torch.cuda.stream(side):
        torch.cuda._sleep(HOLD)
    plan = make()
    sizes = [t.numel() * t.element_size() for t in vars(plan).values() if isinstance(t, torch.Tensor)]
    got = call(plan, side)
    del plan, make, call
    junk = [torch.full((n,), 255, dtype=torch.uint8, device="cuda")
            for n in sizes + [2 * N * w * HD for w in (HEADS, KV, KV, HEADS)] for _ in range(2)]
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    del junk


def test_lens_moves_on_behind_the_step():
    q, k, v, _ = _rows(2, 3)
    a, b = _decoder(700), _decoder(700)
    want = []
    for _ in range(3):
        want.append(a.step(q, k, v))
        a.advance()
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    got = []
    for _ in range(3):
        with torch.cuda.stream(side):
            torch.cuda._sleep(HOLD // 3)
        got.append(b.step(q, k, v, stream=side))
        b.advance()
    b.step(q, k, v, stream=side)
    b.reset()
    torch.cuda.synchronize()
    assert all(torch.equal(x, y) for x, y in zip(got, want)) and not b.lens.any()


def test_the_current_stream_by_name_and_in_a_capture():
    make, call = _plans()["attention"]
    plan = make()
    want = call(plan, None)
    for s in (torch.cuda.current_stream(), torch.cuda.current_stream().cuda_stream, torch.cuda.default_stream()):
        assert all(torch.equal(x, y) for x, y in zip(call(plan, s), want))
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        got = call(plan, torch.cuda.default_stream())            # back on the default stream
    torch.cuda.synchronize()
    assert all(torch.equal(x, y) for x, y in zip(got, want))
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=side):
        got = call(plan, side)
    for t in got:
        t.fill_(float("nan"))
    g.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(x, y) for x, y in zip(got, want))
    g = torch.cuda.CUDAGraph()
    fork = torch.cuda.Stream()
    with torch.cuda.graph(g, stream=side):
        got = call(plan, fork)                                   # a branch of the capture, joined again
        side.wait_stream(fork)
    for t in got:
        t.fill_(float("nan"))
    g.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(x, y) for x, y in zip(got, want))


def test_steps_on_a_branch_of_a_capture():
    """The branch is joined by the call; lens moves on behind it in the graph, and eagerly afterwards."""
    q, k, v, _ = _rows(2, 5)
    a, b = _decoder(700), _decoder(700)
    want = []
    for _ in range(3):
        want.append(a.step(q, k, v))
        a.advance()
    side, fork = torch.cuda.Stream(), torch.cuda.Stream()
    b.step(q, k, v)                                  # rows 700 are written again by the graph
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=side):
        o = b.step(q, k, v, stream=fork)
        b.advance()
    for w in want[:2]:
        o.fill_(float("nan"))
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(o, w)
    assert torch.equal(b.step(q, k, v, stream=fork), want[2])
    b.advance()
    torch.cuda.synchronize()
    assert torch.equal(b.lens, a.lens)


@pytest.mark.parametrize("tokens", [1, 24])
def test_the_next_call_waits_for_one_on_a_stream_of_its_own(tokens):
    """Steps that share counters and parts, the first of each pair held back on its stream."""
    rows = [_rows(2 * tokens, s)[:3] for s in (6, 7, 8)]
    a, b = _decoder(3500, tokens), _decoder(3500, tokens)
    want = [a.step(*r) for r in rows]
    sides = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    got = []
    for r, s in zip(rows, (sides[0], None, sides[1])):
        if s is not None:
            with torch.cuda.stream(s):
                torch.cuda._sleep(HOLD // 2)
        got.append(b.step(*r, stream=s))
    torch.cuda.synchronize()
    assert all(torch.equal(x, y) for x, y in zip(got, want))
