"""Refusals of the checks of waits that run out, on the host: no case reaches a kernel."""
import pytest

lib_mod = pytest.importorskip("sparse_expert_gb300._lib")
lib = lib_mod.lib

INVALID, UNSUPPORTED, WORKSPACE = 1, 2, 6
FAKE, BIG = 1 << 20, 1 << 40  # never dereferenced


@pytest.mark.parametrize("status,bad", [
    (INVALID, dict(limit=0)), (INVALID, dict(limit=-1)), (INVALID, dict(limit=2_000_000_001)), (INVALID, dict(spoiled=-2)),
    # 4 * 2 units at most and 128 / 32 strips
    (INVALID, dict(spoiled=12)), (WORKSPACE, dict(spoiled=11, ws=None)), (UNSUPPORTED, dict(T=65)), (INVALID, dict(x=None))])
def test_few(status, bad):
    a = {**dict(x=FAKE, T=4, ws=FAKE, spoiled=-1, limit=1000), **bad}
    assert lib.moe_selftest_few_wait(a["x"], FAKE, FAKE, 0, 128, a["T"], 128, 8, 2, 128, FAKE, a["ws"], BIG, a["spoiled"],
                                     a["limit"], None) == status


@pytest.mark.parametrize("status,bad", [
    (INVALID, dict(limit=0)), (INVALID, dict(limit=2_000_000_001)), (INVALID, dict(strips=-1)), (UNSUPPORTED, dict(M=17)),
    (INVALID, dict(x=None))])
def test_linear(status, bad):
    a = {**dict(x=FAKE, M=2, strips=0, limit=1000), **bad}
    assert lib.moe_selftest_linear_int4_wait(a["x"], 128, FAKE, a["M"], 128, 64, 64, FAKE, 64, a["strips"], a["limit"],
                                             None) == status
