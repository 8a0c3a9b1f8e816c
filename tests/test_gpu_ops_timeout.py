"""Failure path of fm_gemm_e4m3_b128: a warp of the pipeline gives up
(fm_ops_test_stall), every other wait runs out its short bound, and the call ends
by itself, is reported by fm_ops_sync and leaves the device as it was.  No wait
needs the long bound of a kernel's end: what is in flight there has arrived."""
import threading
import time

import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("no CUDA device", allow_module_level=True)

from vla_flow_matching_denoise_b200 import ops  # noqa: E402
from vla_flow_matching_denoise_b200.binding import FmError, load  # noqa: E402

TMA0, TMA1, MMA0, MMA1 = 1, 2, 3, 4
SPIN = 20000                # cycles: about 10 us

# m, n, k, groups of 128 inputs a block owns, whether a second block (or MMA warp) owns some too
CASES = [(16, 19000, 2048, 16, False),        # a tile per block
         (50, 8192, 2048, 8, True),           # two blocks of a cluster split k
         (50, 1024, 16384, 16, True),         # eight
         (300, 18944, 1024, 16, True),        # a pair of blocks, two tiles for each
         (2500, 4096, 2048, 32, True)]


class _Stall:
    def __init__(self, role, group, spin=SPIN):
        self.args = (role, group, spin)

    def __enter__(self):
        assert load().fm_ops_test_stall(*self.args) == 0

    def __exit__(self, *_):
        assert load().fm_ops_test_stall(0, 0, 0) == 0


def _operands(m, n, k):
    g = torch.Generator(device="cuda").manual_seed(m + n + k)
    a, sa = ops.gated_e4m3(torch.randn(m, k, generator=g, device="cuda"), "none")
    w, sw = ops.quantize_weight_e4m3((torch.randn(n, k, generator=g, device="cuda") * 0.05).bfloat16())
    return a, sa, w, sw


@pytest.mark.parametrize("m,n,k,groups,second", CASES)
@pytest.mark.parametrize("role", [TMA0, TMA1, MMA0, MMA1])
def test_a_role_that_gives_up(m, n, k, groups, second, role):
    ins = _operands(m, n, k)
    want = ops.gemm_e4m3(*ins)
    ops.sync()
    for group in sorted({0, 1, 2, 4, 5, 6, 7, groups - 1}):
        if group >= groups:
            continue
        buf = torch.full((m + 2, n), 7.0, device="cuda", dtype=torch.bfloat16)
        torch.cuda.synchronize()
        t0 = time.perf_counter()
        with _Stall(role, group):
            ops.gemm_e4m3(*ins, out=buf[1:m + 1])
        if second or role in (TMA0, MMA0):
            with pytest.raises(FmError, match="gave up") as e:
                ops.sync()
            assert e.value.status == 5
            assert time.perf_counter() - t0 < 1.0       # the long bound alone is about 2 s
        else:
            assert torch.equal(buf[1:m + 1], want)
        assert torch.all(buf[0] == 7) and torch.all(buf[m + 1] == 7)
        ops.sync()                                      # reported once
        assert torch.equal(ops.gemm_e4m3(*ins), want)
        ops.sync()


@pytest.mark.parametrize("m,n,k,groups,second", CASES)
def test_a_role_past_its_work_changes_nothing(m, n, k, groups, second):
    ins = _operands(m, n, k)
    want = ops.gemm_e4m3(*ins)
    for role in (TMA0, TMA1, MMA0, MMA1):
        with _Stall(role, 4096, 0):
            assert torch.equal(ops.gemm_e4m3(*ins), want)
    ops.sync()


def test_a_captured_product_that_gives_up():
    """A graph keeps the bounds it was captured with, and a replay reports as a call does."""
    ins = _operands(40, 1000, 2048)
    want = ops.gemm_e4m3(*ins)
    graph = torch.cuda.CUDAGraph()
    with _Stall(MMA0, 0):
        with torch.cuda.graph(graph):
            out = ops.gemm_e4m3(*ins)
    ops.sync()
    for _ in range(2):
        graph.replay()
        with pytest.raises(FmError, match="gave up"):
            ops.sync()
    del graph, out
    assert torch.equal(ops.gemm_e4m3(*ins), want)
    ops.sync()


def _in_thread(f):
    got = []

    def body():
        try:
            got.append(f())
        except Exception as e:  # noqa: BLE001  (handed to the caller)
            got.append(e)
    t = threading.Thread(target=body)
    t.start()
    t.join()
    return got[0]


def test_every_thread_is_told():
    """A report to one thread takes nothing from another, on its own stream or not."""
    ins = _operands(40, 1000, 2048)
    ops.sync()
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    with _Stall(TMA0, 1):
        ops.gemm_e4m3(*ins, stream=side)
    first = _in_thread(lambda: ops.sync(side))
    assert isinstance(first, FmError) and first.status == 5
    with pytest.raises(FmError, match="gave up"):
        ops.sync()
    ops.sync(side)
    ops.sync(side.cuda_stream)


def test_sync_leaves_captures_alone():
    ins = _operands(40, 1000, 2048)
    want = ops.gemm_e4m3(*ins)
    ops.sync()
    other = torch.cuda.Stream()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        with pytest.raises(FmError, match="being captured"):
            ops.sync()                                  # the captured stream itself
        def elsewhere():
            try:
                ops.sync(other)                         # a thread's first: what gave up before is told
            except FmError as e:
                assert e.status == 5
            ops.sync(other)
        assert _in_thread(elsewhere) is None
        out = ops.gemm_e4m3(*ins)
    graph.replay()
    ops.sync()
    assert torch.equal(out, want)
