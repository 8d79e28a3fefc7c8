"""The entry points of the layer for a few tokens and of 4-bit weights on the host: argument checks and sizes.  No case
reaches a kernel: every call fails host validation before any CUDA call."""
import pytest

lib_mod = pytest.importorskip("sparse_expert_gb300._lib")
lib = lib_mod.lib

OK, INVALID, UNSUPPORTED, CUDA, TIMEOUT, BAD_INDEX, WORKSPACE, NO_DEVICE = range(8)
BF16, FP8, INT4 = range(3)
FAKE = 1 << 20      # never dereferenced: every use below fails validation first
BIG = 1 << 40


def few(x=FAKE, route=FAKE, packed=FAKE, kind=BF16, group=128, T=4, d=128, E=8, k=2, f=128, out=FAKE, idx=None, w=None, ws=FAKE,
        n=BIG, entry="moe_forward_few"):
    return getattr(lib, entry)(x, route, packed, kind, group, T, d, E, k, f, 1, out, idx, w, ws, n, None)


@pytest.mark.parametrize("entry", ["moe_forward_few", "moe_forward_few_routed"])
@pytest.mark.parametrize("status,bad", [
    (INVALID, dict(T=-1)), (UNSUPPORTED, dict(T=65)), (UNSUPPORTED, dict(T=1 << 40)), (UNSUPPORTED, dict(E=0)),
    (UNSUPPORTED, dict(E=1025)), (UNSUPPORTED, dict(k=0)), (UNSUPPORTED, dict(k=9)), (UNSUPPORTED, dict(E=64, k=33)),
    (UNSUPPORTED, dict(d=96)), (UNSUPPORTED, dict(d=0)), (UNSUPPORTED, dict(d=65600)), (UNSUPPORTED, dict(f=96)),
    (UNSUPPORTED, dict(f=65600)), (UNSUPPORTED, dict(kind=3)), (UNSUPPORTED, dict(kind=-1)),
    (UNSUPPORTED, dict(kind=FP8, d=192)), (UNSUPPORTED, dict(kind=FP8, f=64)), (UNSUPPORTED, dict(kind=INT4, d=64)),
    (UNSUPPORTED, dict(kind=INT4, f=192)), (UNSUPPORTED, dict(kind=INT4, group=16)), (UNSUPPORTED, dict(kind=INT4, group=0)),
    (INVALID, dict(packed=None)), (INVALID, dict(x=None)), (INVALID, dict(route=None)), (INVALID, dict(out=None)),
    (INVALID, dict(x=FAKE + 8)), (INVALID, dict(out=FAKE + 2)), (INVALID, dict(route=FAKE + 2)), (INVALID, dict(packed=FAKE + 8)),
    (INVALID, dict(kind=FP8, packed=FAKE + 16)), (INVALID, dict(kind=INT4, packed=FAKE + 128)), (INVALID, dict(idx=FAKE + 2)),
    (INVALID, dict(w=FAKE + 1)), (WORKSPACE, dict(ws=None)), (WORKSPACE, dict(ws=FAKE + 16)),
    (WORKSPACE, dict(n=lib.moe_forward_few_workspace_bytes(4, 8, 2, 128, 128) - 1))])
def test_few_arguments(entry, status, bad):
    assert few(entry=entry, **bad) == status
    assert lib.moe_last_error()


def test_routed_takes_512_experts():
    assert few(entry="moe_forward_few_routed", E=513) == UNSUPPORTED


def test_few_workspace():
    size = lib.moe_forward_few_workspace_bytes
    for bad in ((65, 8, 2, 128, 128), (-1, 8, 2, 128, 128), (4, 8, 9, 128, 128), (4, 8, 2, 100, 128), (4, 8, 2, 128, 32)):
        assert size(*bad) == 0
    assert 256 <= size(0, 8, 2, 128, 128) < size(1, 8, 2, 128, 128) < size(64, 8, 2, 128, 128)
    assert size(64, 1024, 32, 65536, 65536) > 64 * 32 * 65536 * 6


@pytest.mark.parametrize("status,bad", [
    (INVALID, dict(n=-1)), (UNSUPPORTED, dict(n=65537)), (UNSUPPORTED, dict(K=12)), (UNSUPPORTED, dict(K=0)),
    (UNSUPPORTED, dict(K=65544)), (UNSUPPORTED, dict(N=0)), (UNSUPPORTED, dict(N=(1 << 24) + 1)), (UNSUPPORTED, dict(group=100)),
    (INVALID, dict(w=None)), (INVALID, dict(codes=None)), (INVALID, dict(scales=None)), (INVALID, dict(w=FAKE + 1)),
    (INVALID, dict(scales=FAKE + 1))])
def test_quantize_arguments(status, bad):
    a = {**dict(w=FAKE, n=1, K=128, N=64, group=64, codes=FAKE, scales=FAKE), **bad}
    assert lib.moe_quantize_int4(a["w"], a["n"], a["K"], a["N"], a["group"], a["codes"], a["scales"], None) == status


def test_quantize_nothing():
    assert lib.moe_quantize_int4(None, 0, 128, 64, 64, None, None, None) == OK


@pytest.mark.parametrize("status,bad", [
    (UNSUPPORTED, dict(E=0)), (UNSUPPORTED, dict(E=1025)), (UNSUPPORTED, dict(d=64)), (UNSUPPORTED, dict(f=200)),
    (UNSUPPORTED, dict(group=256)), (INVALID, dict(p=FAKE + 128)), (INVALID, dict(p=None)), (INVALID, dict(c=None)),
    (INVALID, dict(s=FAKE + 1))])
def test_pack_weights_arguments(status, bad):
    a = {**dict(c=FAKE, s=FAKE, E=4, d=128, f=128, group=64, p=FAKE), **bad}
    assert lib.moe_pack_weights_int4(a["c"], a["s"], FAKE, FAKE, FAKE, FAKE, a["E"], a["d"], a["f"], a["group"], a["p"],
                                     None) == status


def test_packed_sizes():
    assert lib.moe_int4_packed_weight_bytes(4, 64, 128, 128) == 0
    # 4-bit codes and a bf16 scale for each group, nothing else where sizes are whole records
    assert lib.moe_int4_packed_weight_bytes(3, 256, 128, 32) == 3 * 3 * 256 * 128 // 2 + 3 * 3 * 256 * 128 // 32 * 2
    assert lib.moe_linear_int4_packed_bytes(256, 128, 64) == 256 * 128 // 2 + 256 * 128 // 64 * 2
    assert lib.moe_linear_int4_packed_bytes(8, 1, 64) == 64 * 128 // 2 + 64 * 2 * 2
    assert lib.moe_linear_int4_packed_bytes(12, 1, 64) == 0 == lib.moe_linear_int4_packed_bytes(16, 1, 63)


@pytest.mark.parametrize("status,bad", [
    (UNSUPPORTED, dict(K=100)), (UNSUPPORTED, dict(N=0)), (UNSUPPORTED, dict(group=0)), (INVALID, dict(c=None)),
    (INVALID, dict(s=FAKE + 1)), (INVALID, dict(p=FAKE + 64))])
def test_pack_linear_arguments(status, bad):
    a = {**dict(c=FAKE, s=FAKE, K=128, N=64, group=64, p=FAKE), **bad}
    assert lib.moe_pack_linear_int4(a["c"], a["s"], a["K"], a["N"], a["group"], a["p"], None) == status


@pytest.mark.parametrize("status,bad", [
    (INVALID, dict(M=-1)), (UNSUPPORTED, dict(M=17)), (UNSUPPORTED, dict(K=100)), (UNSUPPORTED, dict(N=-5)),
    (UNSUPPORTED, dict(group=1)), (INVALID, dict(x=None)), (INVALID, dict(p=None)), (INVALID, dict(out=None)),
    (INVALID, dict(xs=120)), (INVALID, dict(os=63)), (INVALID, dict(x=FAKE + 2)), (INVALID, dict(xs=132)),
    (INVALID, dict(p=FAKE + 16)), (INVALID, dict(out=FAKE + 1))])
def test_linear_arguments(status, bad):
    a = {**dict(x=FAKE, xs=128, p=FAKE, M=2, K=128, N=64, group=64, out=FAKE, os=64), **bad}
    assert lib.moe_linear_int4(a["x"], a["xs"], a["p"], a["M"], a["K"], a["N"], a["group"], a["out"], a["os"], None) == status


def test_linear_of_no_rows():
    assert lib.moe_linear_int4(None, 0, None, 0, 128, 64, 64, None, 0, None) == OK
