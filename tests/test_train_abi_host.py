"""The training-step entry points on the host: argument checks and the
optimizer's coefficients.  No case reaches a kernel: every call fails host
validation before any CUDA call, or is host arithmetic only.
"""
import ctypes
import math

import pytest

lib_mod = pytest.importorskip("sparse_expert_gb300._lib")
lib = lib_mod.lib

OK, INVALID, UNSUPPORTED, CUDA, TIMEOUT, BAD_INDEX, WORKSPACE, NO_DEVICE = range(8)
F32, BF16, F16 = range(3)
FAKE = 1 << 20      # never dereferenced: every use below fails validation first
ODD = FAKE + 1
BIG = 1 << 30


def norm(x=FAKE, xs=64, res=None, rs=0, w=FAKE, b=FAKE, T=4, d=64, dt=BF16, wdt=F32, eps=1e-5, y=FAKE, z=None,
         stats=FAKE):
    return lib.moe_layer_norm(x, xs, res, rs, w, b, T, d, dt, wdt, eps, y, z, stats, None)


@pytest.mark.parametrize("status,bad", [
    (INVALID, dict(T=-1)), (UNSUPPORTED, dict(T=1 << 31)), (UNSUPPORTED, dict(d=0)), (UNSUPPORTED, dict(d=65537)),
    (UNSUPPORTED, dict(dt=3)), (UNSUPPORTED, dict(dt=-1)), (UNSUPPORTED, dict(wdt=F16)), (INVALID, dict(eps=-1e-6)),
    (INVALID, dict(eps=float("nan"))), (INVALID, dict(x=None)), (INVALID, dict(y=None)), (INVALID, dict(stats=None)),
    (INVALID, dict(xs=63)), (INVALID, dict(xs=-64)), (INVALID, dict(x=ODD)), (INVALID, dict(y=ODD)),
    (INVALID, dict(w=FAKE + 2)), (INVALID, dict(stats=FAKE + 2)), (INVALID, dict(z=FAKE)),
    (INVALID, dict(res=FAKE, rs=64)), (INVALID, dict(res=FAKE, rs=63, z=FAKE)), (INVALID, dict(res=ODD, rs=64, z=FAKE))])
def test_layer_norm_arguments(status, bad):
    assert norm(**bad) == status
    assert lib.moe_last_error()


def test_layer_norm_of_no_rows_needs_nothing():
    assert norm(T=0, x=None, y=None, stats=None) == OK


def norm_bwd(dy=FAKE, dys=64, z=FAKE, zs=64, stats=FAKE, w=FAKE, dz=None, dzs=0, T=4, d=64, dt=BF16, wdt=F32, dx=FAKE,
             dw=FAKE, db=FAKE, ws=FAKE, n=BIG):
    return lib.moe_layer_norm_backward(dy, dys, z, zs, stats, w, dz, dzs, T, d, dt, wdt, dx, dw, db, ws, n, None)


@pytest.mark.parametrize("status,bad", [
    (INVALID, dict(T=-1)), (UNSUPPORTED, dict(d=65537)), (UNSUPPORTED, dict(dt=7)), (UNSUPPORTED, dict(wdt=F16)),
    (INVALID, dict(dy=None)), (INVALID, dict(z=None)), (INVALID, dict(stats=None)), (INVALID, dict(dx=None)),
    (INVALID, dict(dys=10)), (INVALID, dict(zs=10)), (INVALID, dict(dz=FAKE, dzs=10)), (INVALID, dict(dx=ODD)),
    (INVALID, dict(dw=FAKE + 2)), (WORKSPACE, dict(ws=None)), (WORKSPACE, dict(ws=FAKE + 16)),
    (WORKSPACE, dict(n=lib.moe_layer_norm_backward_workspace_bytes(4, 64) - 1))])
def test_layer_norm_backward_arguments(status, bad):
    assert norm_bwd(**bad) == status


def test_layer_norm_workspace():
    size = lib.moe_layer_norm_backward_workspace_bytes
    assert size(-1, 64) == 0 and size(4, 0) == 0
    assert 0 < size(1, 64) <= size(100, 64) <= size(10 ** 6, 64) == size(10 ** 8, 64)


def router(logits=FAKE, counts=FAKE, mask=None, T=4, E=8, cb=0.1, cz=0.1, d_in=None, d=FAKE, losses=FAKE, ws=FAKE,
           n=BIG):
    return lib.moe_router_loss(logits, counts, mask, T, E, cb, cz, d_in, d, losses, ws, n, None)


@pytest.mark.parametrize("status,bad", [
    (INVALID, dict(T=-1)), (UNSUPPORTED, dict(E=0)), (UNSUPPORTED, dict(E=1025)), (UNSUPPORTED, dict(T=1 << 40)),
    (INVALID, dict(cb=float("inf"))), (INVALID, dict(cz=float("nan"))), (INVALID, dict(logits=None)),
    (INVALID, dict(counts=None)), (INVALID, dict(d=None)), (INVALID, dict(losses=None)), (INVALID, dict(logits=ODD)),
    (INVALID, dict(d_in=ODD)), (INVALID, dict(losses=FAKE + 2)), (WORKSPACE, dict(ws=None)),
    (WORKSPACE, dict(ws=FAKE + 4)), (WORKSPACE, dict(n=16))])
def test_router_loss_arguments(status, bad):
    assert router(**bad) == status


def record(**over):
    r = lib_mod.AdamWTensor(param=FAKE, grad=FAKE, m=FAKE, v=FAKE, n=10, param_type=BF16, grad_type=BF16, state_bits=32,
                            decay=1.0)
    for k, v in over.items():
        setattr(r, k, v)
    return (lib_mod.AdamWTensor * 1)(r)


HYPER = lib_mod.AdamWHyper()
HOST = ctypes.addressof(HYPER)


@pytest.mark.parametrize("status,bad", [
    (INVALID, dict(n=-1)), (UNSUPPORTED, dict(n=1 << 42)), (UNSUPPORTED, dict(param_type=3)),
    (UNSUPPORTED, dict(grad_type=-1)), (UNSUPPORTED, dict(state_bits=16)), (INVALID, dict(param=None)),
    (INVALID, dict(grad=None)), (INVALID, dict(m=None)), (INVALID, dict(v=None)), (INVALID, dict(state_bits=8)),
    (INVALID, dict(state_bits=8, m_scale=FAKE)), (INVALID, dict(decay=-0.5)), (INVALID, dict(decay=float("nan"))),
    (INVALID, dict(param=ODD)), (INVALID, dict(grad=ODD)), (INVALID, dict(master=FAKE + 2)), (INVALID, dict(m=FAKE + 2)),
    (INVALID, dict(state_bits=8, m_scale=FAKE + 1, v_scale=FAKE))])
def test_adamw_records(status, bad):
    assert lib.moe_adamw_step(record(**bad), 1, HOST, None, None, None) == status


@pytest.mark.parametrize("n", [(1 << 42) - 2047, (1 << 42) - 1])
def test_tensors_of_more_chunks_than_numbers(n):
    """Refused: such a tensor fits no launch, and the host would look for one without end."""
    assert lib.moe_adamw_step(record(n=n), 1, HOST, None, None, None) == UNSUPPORTED
    assert lib.moe_grad_norm(record(n=n), 1, 1.0, FAKE, FAKE, BIG, None) == UNSUPPORTED


def test_adamw_arguments():
    r = record()
    assert lib.moe_adamw_step(r, -1, HOST, None, None, None) == INVALID
    assert lib.moe_adamw_step(None, 1, HOST, None, None, None) == INVALID
    assert lib.moe_adamw_step(r, 1, None, None, None, None) == INVALID
    assert lib.moe_adamw_step(r, 1, HOST, FAKE, None, None) == INVALID
    assert lib.moe_adamw_step(r, 1, None, FAKE + 1, None, None) == INVALID
    assert lib.moe_adamw_step(r, 1, HOST, None, FAKE + 1, None) == INVALID


def test_grad_norm_arguments():
    r = record()
    inf = float("inf")
    assert lib.moe_grad_norm(r, -1, inf, FAKE, FAKE, BIG, None) == INVALID
    assert lib.moe_grad_norm(None, 2, inf, FAKE, FAKE, BIG, None) == INVALID
    assert lib.moe_grad_norm(r, 1, 0.0, FAKE, FAKE, BIG, None) == INVALID
    assert lib.moe_grad_norm(r, 1, float("nan"), FAKE, FAKE, BIG, None) == INVALID
    assert lib.moe_grad_norm(r, 1, inf, None, FAKE, BIG, None) == INVALID
    assert lib.moe_grad_norm(r, 1, inf, FAKE, None, BIG, None) == WORKSPACE
    assert lib.moe_grad_norm(r, 1, inf, FAKE, FAKE, 8, None) == WORKSPACE
    assert lib.moe_grad_norm(record(grad=ODD), 1, inf, FAKE, FAKE, BIG, None) == INVALID
    assert lib.moe_grad_norm(record(n=-5), 1, inf, FAKE, FAKE, BIG, None) == INVALID


def test_grad_norm_of_more_tensors_than_partial_sums():
    """A launch takes up to 384 tensors and needs a partial sum of its own."""
    n = 4096 * 384 + 1
    empty = (lib_mod.AdamWTensor * n)()
    assert lib.moe_grad_norm(empty, n, 1.0, FAKE, FAKE, BIG, None) == UNSUPPORTED


@pytest.mark.parametrize("bad", [dict(lr=-1e-3), dict(lr=math.nan), dict(lr=math.inf), dict(b1=1.0), dict(b1=-0.1),
                                 dict(b2=1.0), dict(b2=math.nan), dict(eps=-1.0), dict(wd=math.inf), dict(step=0)])
def test_adamw_hyper_arguments(bad):
    a = {**dict(lr=1e-3, b1=0.9, b2=0.95, eps=1e-8, wd=0.1, step=1), **bad}
    h = lib_mod.AdamWHyper()
    assert lib.moe_adamw_hyper(a["lr"], a["b1"], a["b2"], a["eps"], a["wd"], a["step"], ctypes.byref(h)) == INVALID


@pytest.mark.parametrize("step", [1, 2, 1000, 10 ** 9])
def test_adamw_hyper_values(step):
    h = lib_mod.AdamWHyper()
    assert lib.moe_adamw_hyper(1e-3, 0.9, 0.999, 1e-8, 0.1, step, ctypes.byref(h)) == OK
    want = dict(beta1=0.9, one_minus_beta1=0.1, beta2=0.999, one_minus_beta2=0.001, step_size=1e-3 / (1 - 0.9 ** step),
                decay=1e-4, inv_sqrt_bias=1 / math.sqrt(1 - 0.999 ** step), eps=1e-8)
    for name, v in want.items():
        assert abs(getattr(h, name) - v) <= 2.0 ** -24 * v, name
