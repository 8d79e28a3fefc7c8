"""The router's auxiliary losses and their gradient against 64 bits.

Tolerance: with u = 2^-24, a probability has a relative error of at most
(range + 40) u (the difference to the row's maximum is rounded, up to `range`
in size; the exponential and a sum of up to 32 + 5 additions), the weighted
sum of probabilities the same, and the loss sums over rows `adds` more.
"""
import pytest
import torch

pytestmark = pytest.mark.gpu

U = 2.0 ** -24


@pytest.fixture(scope="module")
def moe():
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    import sparse_expert_gb300 as m
    return m


def inputs(T, E, seed, spread=1.0):
    g = torch.Generator().manual_seed(seed)
    logits = (torch.randn(T, E, generator=g) * spread + torch.randn(E, generator=g)).cuda()
    counts = torch.randint(0, 50, (E,), generator=g).to(torch.int32).cuda()
    counts[0] += 1
    mask = (torch.rand(T, generator=g) > 0.3).cuda()
    return logits, counts, mask


def reference(logits, counts, cb, cz, mask=None, d_in=None):
    """(losses, gradient, tolerances of both)."""
    T, E = logits.shape
    l = logits.double()
    total = counts.double().sum()
    share = counts.double() / total if total > 0 else torch.zeros(E, dtype=torch.float64, device=l.device)
    live = torch.ones(T, dtype=torch.bool, device=l.device) if mask is None else mask.bool()
    n = int(live.sum())
    empty = torch.isneginf(l).all(1)
    use = live & ~empty
    p, lse, s = torch.zeros_like(l), torch.zeros(T, dtype=l.dtype, device=l.device), None
    p[use] = torch.softmax(l[use], 1)
    lse[use] = torch.logsumexp(l[use], 1)
    s = p @ share
    inv = 1.0 / n if n else 0.0
    losses = torch.stack([E * s.sum() * inv, (lse * lse).sum() * inv])
    d = p * inv * (cb * E * (share - s[:, None]) + 2 * cz * lse[:, None])
    finite = torch.where(torch.isfinite(l), l, torch.zeros_like(l))
    span = (finite.amax(1) - finite.amin(1))[:, None]
    rel = (2 * span + 80) * U
    size = p * inv * (abs(cb) * E * (share + s[:, None]) + 2 * abs(cz) * (lse.abs()[:, None] + 1))
    tol = rel * size + 1e-44
    if d_in is not None:
        d = d_in.double() + d
        tol = tol + U * d.abs()
    adds = 64 + T // 64
    tol_l = torch.stack([(rel.max() + adds * U) * losses[0].abs(),
                         (rel.max() * 2 + adds * U) * (losses[1].abs() + (lse.abs().sum() * inv))]) + 1e-44
    return losses, d, tol_l, tol


def check(moe, logits, counts, mask, cb=0.02, cz=0.003, d_in=None):
    want_l, want_d, tol_l, tol_d = reference(logits, counts, cb, cz, mask, d_in)
    acc = d_in.clone() if d_in is not None else None
    losses, d = moe.moe_router_loss(logits, counts, cb, cz, mask=mask, accumulate=acc)
    if acc is not None:
        assert d is acc
    assert torch.all((losses.double() - want_l).abs() <= tol_l), (losses, want_l)
    err = (d.double() - want_d).abs()
    assert torch.all(err <= tol_d), (err - tol_d).max().item()
    return losses, d


@pytest.mark.parametrize("T", [1, 2, 63, 1000])
@pytest.mark.parametrize("E", [1, 2, 3, 8, 31, 32, 33, 64, 100, 128, 129, 255, 384, 500, 512, 700, 1023, 1024])
def test_losses_and_gradient(moe, T, E):
    logits, counts, mask = inputs(T, E, seed=T * 2000 + E)
    check(moe, logits, counts, None)
    check(moe, logits, counts, mask)
    check(moe, logits, counts, mask, d_in=torch.randn(T, E, device="cuda") * 1e-3)


@pytest.mark.parametrize("T,E", [(30000, 8), (20011, 64), (9000, 384), (40000, 5)])
def test_many_rows(moe, T, E):
    logits, counts, mask = inputs(T, E, seed=T)
    check(moe, logits, counts, mask, d_in=torch.randn(T, E, device="cuda") * 1e-5)


@pytest.mark.parametrize("T,E", [(22003, 384), (90001, 64), (13003, 768), (13001, 1000), (13007, 1023)])
def test_more_pieces_than_blocks(moe, T, E):
    """Blocks go on from piece to piece, the last of them partial: every row
    right, and the same bits whichever block takes it."""
    logits, counts, mask = inputs(T, E, seed=T)
    d_in = torch.randn(T, E, device="cuda") * 1e-5
    check(moe, logits, counts, None)
    check(moe, logits, counts, None, d_in=d_in)
    check(moe, logits, counts, mask)
    first = check(moe, logits, counts, mask, d_in=d_in)
    for _ in range(3):
        again = moe.moe_router_loss(logits, counts, 0.02, 0.003, mask=mask, accumulate=d_in.clone())
        assert all(torch.equal(p, q) for p, q in zip(first, again))


@pytest.mark.parametrize("T,E", [(100, 64), (100, 33), (9001, 384), (22003, 384), (30001, 8)])
@pytest.mark.parametrize("masked", [False, True])
def test_gradient_added_to_one_that_stays(moe, T, E, masked):
    """d_in apart from d_logits: read and not written; masked rows are copies of it."""
    logits, counts, mask = inputs(T, E, seed=T + E)
    mask = mask if masked else None
    d_in = torch.randn(T, E, device="cuda") * 1e-4
    kept = d_in.clone()
    d, losses = torch.full_like(logits, float("nan")), torch.empty(2, device="cuda")
    ws = torch.empty(moe._lib.lib.moe_router_loss_workspace_bytes(), dtype=torch.uint8, device="cuda")
    ptr = lambda t: None if t is None else t.data_ptr()  # noqa: E731
    assert moe._lib.lib.moe_router_loss(ptr(logits), ptr(counts), ptr(mask), T, E, 0.02, 0.003, ptr(d_in), ptr(d),
                                        ptr(losses), ptr(ws), ws.numel(),
                                        torch.cuda.current_stream().cuda_stream) == 0
    want_l, want_d, tol_l, tol_d = reference(logits, counts, 0.02, 0.003, mask, d_in)
    assert torch.equal(d_in, kept) and torch.all((d.double() - want_d).abs() <= tol_d)
    assert torch.all((losses.double() - want_l).abs() <= tol_l)
    if masked:
        assert torch.equal(d[~mask], d_in[~mask])


@pytest.mark.parametrize("T,E", [(100, 64), (9001, 384), (22003, 384)])
@pytest.mark.parametrize("masked", [False, True])
def test_graph_replay(moe, T, E, masked):
    logits, counts, mask = inputs(T, E, seed=3)
    mask = mask if masked else None
    out, losses = torch.empty_like(logits), torch.empty(2, device="cuda")
    ws = torch.empty(moe._lib.lib.moe_router_loss_workspace_bytes(), dtype=torch.uint8, device="cuda")
    stream, graph = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.stream(stream):
        with torch.cuda.graph(graph, stream=stream):
            moe.moe_router_loss(logits, counts, mask=mask, out=out, losses=losses, workspace=ws, stream=stream)
    for seed in (4, 5):
        new, new_counts, new_mask = inputs(T, E, seed=seed)
        logits.copy_(new), counts.copy_(new_counts)
        if masked:
            mask.copy_(new_mask)
        graph.replay()
        want_l, want_d = moe.moe_router_loss(new, new_counts, mask=new_mask if masked else None)
        torch.cuda.synchronize()
        assert torch.equal(out, want_d) and torch.equal(losses, want_l)


def test_unaligned_rows(moe):
    buf = torch.randn(200 * 64 + 1, device="cuda")
    logits = buf[1:].view(200, 64)
    counts = torch.arange(64, dtype=torch.int32, device="cuda")
    out = torch.empty(200 * 64 + 3, device="cuda")[3:].view(200, 64)
    want_l, want_d, tol_l, tol_d = reference(logits, counts, 0.5, 0.5)
    mask = torch.cat([torch.zeros(1, dtype=torch.bool), torch.ones(200, dtype=torch.bool)]).cuda()[1:]
    losses, d = moe.moe_router_loss(logits, counts, 0.5, 0.5, mask=mask, out=out)
    assert d is out and torch.all((d.double() - want_d).abs() <= tol_d)
    assert torch.all((losses.double() - want_l).abs() <= tol_l)


def test_wide_range_of_logits(moe):
    logits, counts, mask = inputs(300, 96, seed=9, spread=30.0)
    check(moe, logits, counts, mask)


def test_balanced_routing_has_loss_one(moe):
    losses, _ = moe.moe_router_loss(torch.zeros(40, 16, device="cuda"),
                                    torch.full((16,), 5, dtype=torch.int32, device="cuda"), 1.0, 0.0)
    assert abs(losses[0].item() - 1.0) <= 100 * U


def test_masked_rows_are_not_read_and_get_no_gradient(moe):
    logits, counts, mask = inputs(400, 40, seed=10)
    want = moe.moe_router_loss(logits, counts, mask=mask)
    poisoned = logits.clone()
    poisoned[~mask] = float("nan")
    got = moe.moe_router_loss(poisoned, counts, mask=mask)
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    assert not got[1][~mask].any()
    before = torch.randn(400, 40, device="cuda")
    after = moe.moe_router_loss(poisoned, counts, mask=mask, accumulate=before.clone())[1]
    assert torch.equal(after[~mask], before[~mask])


@pytest.mark.parametrize("T,E,k", [(300, 16, 2), (5001, 384, 8)])
def test_counts_decide_which_rows_make_the_shares(moe, T, E, k):
    """Counts of the kept rows: the losses and gradients of those rows alone.
    Counts of all routed rows: the kept rows against the load with the others."""
    logits, _, mask = inputs(T, E, seed=T)
    topk = torch.topk(logits, k, 1).indices

    def counted(rows):
        return torch.bincount(topk[rows].flatten(), minlength=E).to(torch.int32)
    every, kept = counted(torch.ones_like(mask)), counted(mask)
    assert not torch.equal(every, kept)
    _, d = check(moe, logits, kept, mask)
    _, _, tol_l, tol_d = reference(logits[mask], kept, 0.02, 0.003)
    alone = moe.moe_router_loss(logits[mask], kept, 0.02, 0.003)
    assert torch.all((moe.moe_router_loss(logits, kept, 0.02, 0.003, mask=mask)[0] - alone[0]).abs() <= 2 * tol_l)
    assert torch.all((d[mask] - alone[1]).abs() <= 2 * tol_d)
    with_all, _ = check(moe, logits, every, mask)
    p = torch.softmax(logits[mask].double(), 1).mean(0)
    want = E * (p * every.double() / (T * k)).sum()
    assert abs(with_all[0].item() - want.item()) <= 1e-5 * want.item()


def test_nothing_kept(moe):
    logits, counts, _ = inputs(77, 24, seed=11)
    none = torch.zeros(77, dtype=torch.bool, device="cuda")
    losses, d = moe.moe_router_loss(logits, counts, mask=none)
    assert not losses.any() and not d.any()
    losses, d = moe.moe_router_loss(logits, torch.zeros_like(counts), 0.1, 0.0)
    assert losses[0] == 0 and not d.any()
    losses, d = moe.moe_router_loss(logits[:0], counts)
    assert not losses.any() and d.shape == (0, 24)


def test_experts_and_rows_at_minus_infinity(moe):
    logits, counts, mask = inputs(90, 48, seed=12)
    logits[:, 5] = float("-inf")
    logits[7] = float("-inf")
    logits[8, 1:] = float("-inf")
    lowest = torch.finfo(torch.float32).min
    logits[9, ::2] = lowest
    logits[10] = lowest
    # the span of a row with the type's lowest value is no measure of the error: its probabilities there are zero
    ref_in = torch.where(logits == lowest, torch.full_like(logits, -1e30), logits)
    losses, d = moe.moe_router_loss(logits, counts, 0.02, 0.0)
    rows = [r for r in range(90) if r not in (9, 10)]
    _, want, _, tol = reference(ref_in, counts, 0.02, 0.0)
    assert torch.isfinite(losses[0]) and torch.isfinite(d).all()
    assert torch.all((d.double() - want).abs()[rows] <= tol[rows])
    assert not d[7].any() and not d[:10, 5].any() and not d[11:, 5].any() and not d[9, ::2].any()


@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
def test_a_bad_logit_shows_and_stays_in_its_row(moe, bad):
    logits, counts, _ = inputs(50, 33, seed=13)
    good = moe.moe_router_loss(logits, counts)[1]
    logits[20, 3] = bad
    losses, d = moe.moe_router_loss(logits, counts)
    keep = [t for t in range(50) if t != 20]
    assert torch.isnan(losses).all() and torch.isnan(d[20]).all() and torch.equal(d[keep], good[keep])


def test_gradient_against_differences(moe):
    """Central differences of the 64-bit losses around fp32 logits: truncation h^2, rounding 1e-16 / h."""
    logits, counts, mask = inputs(30, 12, seed=14)
    cb, cz, h = 0.7, 0.2, 1e-4
    d = moe.moe_router_loss(logits, counts, cb, cz, mask=mask)[1].double()

    def loss(l):
        share = counts.double() / counts.double().sum()
        m = mask.double()
        balance = 12 * ((torch.softmax(l, 1) @ share) * m).sum() / m.sum()
        return cb * balance + cz * (torch.logsumexp(l, 1).pow(2) * m).sum() / m.sum()
    l64 = logits.double()
    for t, e in [(0, 0), (3, 7), (12, 11), (25, 4), (29, 2)]:
        step = torch.zeros_like(l64)
        step[t, e] = h
        diff = ((loss(l64 + step) - loss(l64 - step)) / (2 * h)).item()
        assert abs(diff - d[t, e].item()) <= 10 * h * h + 1e-11 + 200 * U * (abs(diff) + 0.1)


def test_same_bits_every_time_and_on_another_stream(moe):
    logits, counts, mask = inputs(5000, 384, seed=15)
    want = moe.moe_router_loss(logits, counts, mask=mask)
    torch.cuda.synchronize()
    for stream in (None, torch.cuda.Stream()):
        got = moe.moe_router_loss(logits, counts, mask=mask, stream=stream)
        torch.cuda.synchronize()
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


def test_refusals(moe):
    logits, counts, mask = inputs(20, 16, seed=16)
    with pytest.raises(TypeError):
        moe.moe_router_loss(logits.half(), counts)
    with pytest.raises(TypeError):
        moe.moe_router_loss(logits, counts.long())
    with pytest.raises(TypeError):
        moe.moe_router_loss(logits, counts, mask=mask.float())
    with pytest.raises(ValueError):
        moe.moe_router_loss(logits, counts[:8])
    with pytest.raises(ValueError):
        moe.moe_router_loss(logits, counts, mask=mask[:8])
    with pytest.raises(ValueError):
        moe.moe_router_loss(logits.t(), counts)
    with pytest.raises(ValueError):
        moe.moe_router_loss(logits, counts, accumulate=logits.clone(), out=logits.clone())
    with pytest.raises(moe.MoEError) as e:
        moe.moe_router_loss(logits, counts, float("nan"))
    assert e.value.status == 1
    with pytest.raises(moe.MoEError) as e:
        moe.moe_router_loss(torch.zeros(2, 1025, device="cuda"), torch.zeros(1025, dtype=torch.int32, device="cuda"))
    assert e.value.status == 2
    with pytest.raises(moe.MoEError) as e:
        moe.moe_router_loss(logits, counts, workspace=torch.empty(256, dtype=torch.uint8, device="cuda"))
    assert e.value.status == 6
