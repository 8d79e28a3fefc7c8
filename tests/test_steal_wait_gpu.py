"""The wait of kernels that take further pieces of work: a block's threads
must come to one outcome, or a piece that only some of them know of is lost.
The GPU is never made to lose an answer; the wait itself is run, on a barrier
that nothing completes and on one completed late."""
import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def moe():
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    import sparse_expert_gb300 as m
    return m


@pytest.mark.parametrize("limit_ns", [1, 1_000_000, 20_000_000])
def test_all_threads_agree(moe, limit_ns):
    never, late = moe.moe_selftest_steal_wait(limit_ns).tolist()
    assert not any(never) and all(v == 1 for v in late)


def test_refusals(moe):
    for limit in (0, 3_000_000_000):
        with pytest.raises(moe.MoEError) as e:
            moe.moe_selftest_steal_wait(limit)
        assert e.value.status == 1


def test_work_goes_on_after_a_wait_that_ran_out(moe):
    x = torch.randn(9001, 2048, device="cuda").to(torch.bfloat16)
    want = moe.moe_layer_norm(x)
    moe.moe_selftest_steal_wait(1_000_000)
    got = moe.moe_layer_norm(x)
    assert all(torch.equal(a, b) for a, b in zip(want, got)) and torch.isfinite(got[1]).all()
