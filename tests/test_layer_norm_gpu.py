"""Layer norm, forward and backward, against the definition in 64 bits.

Tolerances come from the arithmetic: u = 2^-24 for each fp32 operation, a sum
over a row or over rows in fp32 with at most SUM sequential additions a
thread before the trees, and one rounding to the rows' type at the end.
"""
import pytest
import torch

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
SUM = 80                                  # additions on the longest path of a row's sum (64 + log2 1024, and slack)
ROUND = {torch.float32: 2.0 ** -24, torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11}
TINY = {torch.float32: 2.0 ** -149, torch.bfloat16: 2.0 ** -134, torch.float16: 2.0 ** -25}
EPS = 1e-5
DTYPES = [torch.bfloat16, torch.float16, torch.float32]


@pytest.fixture(scope="module")
def moe():
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    import sparse_expert_gb300 as m
    return m


def rows(T, d, dtype, seed, scale=1.0, offset=0.0, stride=None, shift=0):
    """Random rows; with a stride and a shift, a view that starts `shift` values into a larger buffer."""
    g = torch.Generator().manual_seed(seed)
    x = (torch.randn(T, d, generator=g) * scale + offset).to(dtype).cuda()
    if stride is None and shift == 0:
        return x
    stride = stride or d
    buf = torch.full((T * stride + shift + 64,), float("nan"), dtype=dtype, device="cuda")
    view = buf[shift:shift + T * stride].view(T, stride)[:, :d]
    view.copy_(x)
    return view


def params(d, wdtype, seed):
    g = torch.Generator().manual_seed(seed)
    return ((1 + 0.3 * torch.randn(d, generator=g)).to(wdtype).cuda(),
            (0.3 * torch.randn(d, generator=g)).to(wdtype).cuda())


def exact_stats(z, eps=EPS):
    z = z.double()
    mu = z.mean(1)
    return mu, 1.0 / torch.sqrt((z - mu[:, None]).pow(2).mean(1) + eps)


def check_forward(z, w, b, y, stats, eps=EPS):
    """y and stats for the (rounded) rows z against 64 bits."""
    zd = z.double()
    mu, r = exact_stats(z, eps)
    d_mu = SUM * U * zd.abs().mean(1) + U * mu.abs()
    # the variance: a relative error of its sum, and the square of the mean's error; its root halves both
    d_r = r * (0.5 * (SUM + 8) * U + 0.5 * (d_mu * r) ** 2 + 4 * U)
    assert torch.all((stats[0].double() - mu).abs() <= d_mu)
    assert torch.all((stats[1].double() - r).abs() <= d_r)
    e = zd - mu[:, None]
    wd = torch.ones_like(zd[0]) if w is None else w.double()
    bd = torch.zeros_like(zd[0]) if b is None else b.double()
    want = e * r[:, None] * wd + bd
    tol = wd.abs() * (r[:, None] * (d_mu[:, None] + 2 * U * e.abs()) + e.abs() * d_r[:, None])
    tol = tol + 4 * U * (want.abs() + bd.abs()) + ROUND[y.dtype] * want.abs() * 1.01 + TINY[y.dtype]
    err = (y.double() - want).abs()
    assert torch.all(err <= tol), (err - tol).max().item()


SHAPES = [(1, 1), (3, 1), (2, 2), (5, 7), (4, 8), (33, 24), (300, 128), (1, 257), (17, 1001), (64, 1024), (9, 2048),
          (7, 4100), (5, 6144), (3, 8200), (2, 12296), (2, 16384), (3, 20001), (2, 32768), (1, 40007), (2, 65536)]


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("T,d", SHAPES)
def test_forward(moe, T, d, dtype):
    x = rows(T, d, dtype, seed=d)
    w, b = params(d, dtype if d % 2 else torch.float32, seed=1)
    y, stats = moe.moe_layer_norm(x, w, b)
    assert y.dtype == dtype and y.shape == x.shape
    check_forward(x, w, b, y, stats)
    r = rows(T, d, dtype, seed=d + 1, scale=0.5)
    y, stats, z = moe.moe_layer_norm(x, w, b, residual=r)
    assert torch.equal(z, (x.float() + r.float()).to(dtype))
    check_forward(z, w, b, y, stats)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("d,stride,shift", [(64, 80, 0), (128, 131, 0), (128, 128, 1), (257, 257, 3), (1001, 1040, 5),
                                            (2048, 2056, 8), (2048, 2049, 7), (40007, 40010, 1)])
def test_forward_strides_and_alignment(moe, d, stride, shift, dtype):
    x = rows(6, d, dtype, seed=d, stride=stride, shift=shift)
    r = rows(6, d, dtype, seed=d + 1, stride=stride + 3, shift=shift + 2)
    w, b = params(d + 1, torch.float32, seed=2)
    w, b = w[1:], b[1:]                                        # 4-byte aligned parameters
    y, stats = moe.moe_layer_norm(x, w, b)
    check_forward(x, w, b, y, stats)
    out = torch.empty(6 * d + 1, dtype=dtype, device="cuda")[1:].view(6, d)
    y, stats, z = moe.moe_layer_norm(x, w, b, residual=r, out=out)
    assert y is out and torch.equal(z, (x.float() + r.float()).to(dtype))
    check_forward(z, w, b, y, stats)


@pytest.mark.parametrize("residual", [False, True])
@pytest.mark.parametrize("T,d,dtype", [
    (110003, 128, torch.bfloat16), (120011, 136, torch.float16),           # one chunk a thread
    (20003, 1024, torch.bfloat16), (9001, 2048, torch.bfloat16), (5003, 2048, torch.float32),
    (5001, 2056, torch.float16), (2503, 6144, torch.bfloat16), (1203, 16384, torch.bfloat16)])
def test_forward_many_rows(moe, T, d, dtype, residual):
    """More pieces than the SMs hold at once, so that blocks go on from piece
    to piece, the last of them partial: every row right, and the same bits
    whichever block takes it."""
    x = rows(T, d, dtype, seed=T)
    r = rows(T, d, dtype, seed=T + 1, scale=0.5) if residual else None
    w, b = params(d, torch.float32, seed=5)
    first = moe.moe_layer_norm(x, w, b, residual=r)
    z = x
    if residual:
        z = first[2]
        assert torch.equal(z, (x.float() + r.float()).to(dtype))
    check_forward(z, w, b, *first[:2])
    for _ in range(3):
        again = moe.moe_layer_norm(x, w, b, residual=r)
        assert all(torch.equal(p, q) for p, q in zip(first, again))


@pytest.mark.parametrize("w,b", [(False, False), (True, False), (False, True)])
def test_forward_without_weight_or_bias(moe, w, b):
    x = rows(50, 320, torch.bfloat16, seed=3)
    weight, bias = params(320, torch.bfloat16, seed=4)
    weight, bias = weight if w else None, bias if b else None
    y, stats = moe.moe_layer_norm(x, weight, bias)
    check_forward(x, weight, bias, y, stats)


@pytest.mark.parametrize("offset", [100.0, 1e4])
@pytest.mark.parametrize("d", [128, 1001, 6144, 65536])
def test_forward_large_offset(moe, d, offset):
    x = rows(4, d, torch.float32, seed=5, offset=offset)
    x[1, 0] = 3 * offset                                       # the first value far from the rest
    y, stats = moe.moe_layer_norm(x)
    check_forward(x, None, None, y, stats)


def test_forward_constant_rows_and_eps(moe):
    x = torch.full((3, 4096), 1.5, device="cuda")
    x[1] = 0.0
    y, stats = moe.moe_layer_norm(x, eps=0.25)
    assert torch.equal(y, torch.zeros_like(x)) and torch.all(stats[1] == 2.0)
    assert stats[0].tolist() == [1.5, 0.0, 1.5]


@pytest.mark.parametrize("d", [100, 6144, 40000])
@pytest.mark.parametrize("bad", [float("nan"), float("inf"), float("-inf")])
def test_a_bad_value_stays_in_its_row(moe, d, bad):
    x = rows(5, d, torch.bfloat16, seed=6)
    good, _ = moe.moe_layer_norm(x)
    x2 = x.clone()
    x2[2, d // 2] = bad
    y, stats = moe.moe_layer_norm(x2)
    keep = [0, 1, 3, 4]
    assert torch.equal(y[keep], good[keep]) and torch.isnan(y[2]).all()
    dy = rows(5, d, torch.bfloat16, seed=7)
    g = moe.moe_layer_norm_backward(dy, x2, stats, bias=True)
    assert torch.isnan(g["dx"][2]).all() and torch.isfinite(g["dx"][keep]).all() and torch.isfinite(g["dbias"]).all()


def test_no_rows(moe):
    x = torch.empty(0, 96, dtype=torch.bfloat16, device="cuda")
    w, b = params(96, torch.float32, seed=1)
    y, stats = moe.moe_layer_norm(x, w, b)
    assert y.shape == (0, 96) and stats.shape == (2, 0)
    g = moe.moe_layer_norm_backward(x, x, stats, w)
    assert g["dx"].shape == (0, 96) and not g["dweight"].any() and not g["dbias"].any()


# ------------------------------------------------------------------ backward
def check_backward(dy, z, stats, w, dz, got, bias=True):
    T, d = z.shape
    mu, r = stats[0].double()[:, None], stats[1].double()[:, None]
    dyd = dy.double()
    n = (z.double() - mu) * r
    g = dyd if w is None else dyd * w.double()
    s1, s2 = g.mean(1, keepdim=True), (g * n).mean(1, keepdim=True)
    want = r * (g - s1 - n * s2)
    tol = r * (8 * U * (g.abs() + s1.abs() + (n * s2).abs())
               + SUM * U * (g.abs().mean(1, keepdim=True) + n.abs() * (g * n).abs().mean(1, keepdim=True)))
    if dz is not None:
        want = want + dz.double()
    tol = tol + U * want.abs() + ROUND[dy.dtype] * want.abs() * 1.01 + TINY[dy.dtype]
    err = (got["dx"].double() - want).abs()
    assert got["dx"].dtype == dy.dtype and torch.all(err <= tol), (err - tol).max().item()
    adds = 64 + T // 16                    # sequential additions over rows on the longest path
    for name, terms in (("dweight", dyd * n), ("dbias", dyd)):
        if got[name] is None:
            assert name == "dweight" and w is None or name == "dbias" and not bias
            continue
        tol = (adds + 4) * U * terms.abs().sum(0)
        err = (got[name].double() - terms.sum(0)).abs()
        assert got[name].dtype == torch.float32 and torch.all(err <= tol), (name, (err - tol).max().item())


def backward_case(moe, T, d, dtype, wdtype, residual, seed, stride=None, shift=0):
    z = rows(T, d, dtype, seed=seed, offset=0.5, stride=stride, shift=shift)
    dy = rows(T, d, dtype, seed=seed + 1, scale=0.1, stride=stride and stride + 1, shift=shift)
    dz = rows(T, d, dtype, seed=seed + 2, scale=0.1, stride=stride, shift=shift and shift + 1) if residual else None
    w, _ = params(d, wdtype, seed=seed + 3)
    mu, r = exact_stats(z)
    stats = torch.stack([mu, r]).float()
    got = moe.moe_layer_norm_backward(dy, z, stats, w, dz=dz)
    check_backward(dy, z, stats, w, dz, got)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("T,d", SHAPES)
def test_backward(moe, T, d, dtype):
    backward_case(moe, T, d, dtype, dtype if d % 2 else torch.float32, residual=d % 3 != 0, seed=d)


@pytest.mark.parametrize("T,d", [(3000, 64), (2999, 130), (2500, 333), (1200, 2048), (700, 6144), (130, 8192),
                                 (300, 20000), (2000, 5)])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_backward_many_rows(moe, T, d, dtype):
    backward_case(moe, T, d, dtype, torch.float32, residual=True, seed=T)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("d,stride,shift", [(64, 80, 0), (128, 131, 0), (128, 128, 1), (1001, 1040, 5), (2048, 2056, 8),
                                            (2048, 2049, 7), (40007, 40010, 1)])
def test_backward_strides_and_alignment(moe, d, stride, shift, dtype):
    backward_case(moe, 40, d, dtype, torch.float32, residual=True, seed=d, stride=stride, shift=shift)


@pytest.mark.parametrize("T,d,dtype,offset", [
    (T, 6145, dtype, 0) for dtype in (torch.bfloat16, torch.float16) for T in (33, 41, 151)
] + [(33, 3073, torch.float32, 0), (151, 3073, torch.float32, 0), (77, 6144, torch.bfloat16, 1), (60, 16001, torch.float16, 0),
     (93, 2049, torch.bfloat16, 0), (93, 20001, torch.bfloat16, 0), (93, 1001, torch.float32, 1)])
def test_backward_stays_in_its_workspace(moe, T, d, dtype, offset):
    """Rows off a chunk (or, with an offset, weights off 16 bytes), no multiple
    of a chunk's values of them: what lies behind the workspace is not touched."""
    z, dy = rows(T, d, dtype, seed=T, offset=0.5), rows(T, d, dtype, seed=T + 1, scale=0.1)
    w = params(d + offset, torch.float32, seed=3)[0][offset:]
    stats = torch.stack(exact_stats(z)).float()
    size = moe.moe_layer_norm_backward_workspace_bytes(T, d)
    buf = torch.full((size + (4 << 20),), 0xA5, dtype=torch.uint8, device="cuda")
    got = moe.moe_layer_norm_backward(dy, z, stats, w, workspace=buf[:size])
    check_backward(dy, z, stats, w, None, got)
    assert torch.all(buf[size:] == 0xA5)


@pytest.mark.parametrize("weight,bias", [(False, False), (True, False), (False, True)])
@pytest.mark.parametrize("d", [192, 30000])
def test_backward_optional_outputs(moe, weight, bias, d):
    z, dy = rows(70, d, torch.float16, seed=1), rows(70, d, torch.float16, seed=2)
    w = params(d, torch.float16, seed=3)[0] if weight else None
    stats = torch.stack(exact_stats(z)).float()
    got = moe.moe_layer_norm_backward(dy, z, stats, w, bias=bias)
    assert (got["dweight"] is not None) == weight and (got["dbias"] is not None) == bias
    check_backward(dy, z, stats, w, None, got, bias)


@pytest.mark.parametrize("d", [96, 1001, 6144])
def test_gradients_against_differences(moe, d):
    """<dx, v>, <dw, v> and <db, v> against central differences of the fp32
    forward.  With rows of unit size the third derivative along v is of the
    order of the first, so a step h leaves h^2; the forward's rounding leaves
    about u sqrt(T d) / h of the loss's size."""
    T, h = 24, 1e-2
    x, dy, vx = (rows(T, d, torch.float32, seed=s) for s in (1, 2, 3))
    w, b = params(d, torch.float32, seed=4)
    vw, vb = params(d, torch.float32, seed=5)
    y, stats = moe.moe_layer_norm(x, w, b)
    g = moe.moe_layer_norm_backward(dy, x, stats, w)

    def loss(xx, ww, bb):
        return (moe.moe_layer_norm(xx, ww, bb)[0].double() * dy.double()).sum().item()
    size = (T * d) ** 0.5
    tol = 5 * h * h * size + 8 * U * size * 4 / h
    assert abs((loss(x + h * vx, w, b) - loss(x - h * vx, w, b)) / (2 * h) -
               (g["dx"].double() * vx.double()).sum().item()) <= tol
    assert abs((loss(x, w + h * vw, b) - loss(x, w - h * vw, b)) / (2 * h) -
               (g["dweight"].double() * vw.double()).sum().item()) <= tol
    assert abs((loss(x, w, b + h * vb) - loss(x, w, b - h * vb)) / (2 * h) -
               (g["dbias"].double() * vb.double()).sum().item()) <= tol


@pytest.mark.parametrize("T,d", [(4000, 512), (900, 6144), (777, 1001), (90, 30000)])
def test_same_bits_every_time_and_on_another_stream(moe, T, d):
    x, dy, r = (rows(T, d, torch.bfloat16, seed=s) for s in (1, 2, 3))
    w, b = params(d, torch.float32, seed=4)
    y, stats, z = moe.moe_layer_norm(x, w, b, residual=r)
    first = moe.moe_layer_norm_backward(dy, z, stats, w, dz=r)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    for stream in (None, s):
        y2, stats2, z2 = moe.moe_layer_norm(x, w, b, residual=r, stream=stream)
        again = moe.moe_layer_norm_backward(dy, z2, stats2, w, dz=r, stream=stream)
        torch.cuda.synchronize()
        assert torch.equal(y, y2) and torch.equal(stats, stats2) and torch.equal(z, z2)
        assert all(torch.equal(first[k], again[k]) for k in first)


@pytest.mark.parametrize("T,d", [(20, 128), (2503, 6144), (777, 1001), (40, 30000)])
def test_graph_replay(moe, T, d):
    """Forward and backward in one captured graph, replayed on other inputs."""
    x, r, dy = (rows(T, d, torch.bfloat16, seed=s) for s in (1, 2, 3))
    w, b = params(d, torch.float32, seed=4)
    y, z, stats = torch.empty_like(x), torch.empty_like(x), torch.empty(2, T, device="cuda")
    grads = dict(dx=torch.empty_like(x), dweight=torch.empty_like(w), dbias=torch.empty_like(b))
    ws = torch.empty(moe.moe_layer_norm_backward_workspace_bytes(T, d), dtype=torch.uint8, device="cuda")
    stream, graph = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.stream(stream):
        with torch.cuda.graph(graph, stream=stream):
            moe.moe_layer_norm(x, w, b, residual=r, out=y, stats=stats, z=z, stream=stream)
            moe.moe_layer_norm_backward(dy, z, stats, w, dz=r, grads=grads, workspace=ws, stream=stream)
    for seed in (5, 6):
        for t in (x, r, dy):
            t.copy_(rows(T, d, torch.bfloat16, seed=seed))
        graph.replay()
        want = moe.moe_layer_norm(x, w, b, residual=r)
        want_grads = moe.moe_layer_norm_backward(dy, want[2], want[1], w, dz=r)
        torch.cuda.synchronize()
        assert all(torch.equal(p, q) for p, q in zip((y, stats, z), want))
        assert all(torch.equal(grads[k], want_grads[k]) for k in grads)


def test_offsets_beyond_32_bits(moe):
    """Rows whose element offsets pass 2^32: the last rows are right."""
    T, d = 9, 1 << 29
    buf = torch.zeros(T * d, dtype=torch.bfloat16, device="cuda")
    x = buf.view(T, d)[:, :640]                                # row stride 2^29 elements
    x.copy_(rows(T, 640, torch.bfloat16, seed=1))
    y, stats = moe.moe_layer_norm(x)
    check_forward(x, None, None, y, stats)
    g = moe.moe_layer_norm_backward(x, x, stats)
    check_backward(x, x, stats, None, None, g)


def test_refusals(moe):
    x = rows(4, 64, torch.bfloat16, seed=1)
    w, b = params(64, torch.float32, seed=2)
    _, stats = moe.moe_layer_norm(x, w, b)
    with pytest.raises(TypeError):
        moe.moe_layer_norm(x.double())
    with pytest.raises(TypeError):
        moe.moe_layer_norm(x, w.half())
    with pytest.raises(TypeError):
        moe.moe_layer_norm(x, w, b.bfloat16())
    with pytest.raises(TypeError):
        moe.moe_layer_norm(x, residual=x.float())
    with pytest.raises(ValueError):
        moe.moe_layer_norm(x.cpu())
    with pytest.raises(ValueError):
        moe.moe_layer_norm(x.t())
    with pytest.raises(ValueError):
        moe.moe_layer_norm(x[0])
    with pytest.raises(ValueError):
        moe.moe_layer_norm(x, w[:32])
    with pytest.raises(ValueError):
        moe.moe_layer_norm(x, residual=x[:2])
    with pytest.raises(ValueError):
        moe.moe_layer_norm(x, z=torch.empty_like(x))
    with pytest.raises(moe.MoEError) as e:
        moe.moe_layer_norm(x, eps=-1.0)
    assert e.value.status == 1
    with pytest.raises(moe.MoEError) as e:
        moe.moe_layer_norm(torch.zeros(1, 65537, device="cuda"))
    assert e.value.status == 2
    with pytest.raises(moe.MoEError) as e:                    # rows on top of one another
        moe.moe_layer_norm(torch.zeros(100, device="cuda").as_strided((3, 64), (16, 1)))
    assert e.value.status == 1
    with pytest.raises(ValueError):
        moe.moe_layer_norm_backward(x, x, stats[:, :3].contiguous(), w)
    with pytest.raises(moe.MoEError) as e:
        moe.moe_layer_norm_backward(x, x, stats, w, workspace=torch.empty(256, dtype=torch.uint8, device="cuda"))
    assert e.value.status == 6
