"""How calls of one feed-forward handle share its workspace: stream captures,
calls of several streams, tiles that are split, and what a timeout leaves.

Values are compared with the same call made alone, bit for bit: the sums are
taken in a fixed order."""

import threading

import pytest
import torch

from test_gpu_gated_ff import make

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    from gptq_qqq_calibration_gb300 import build as b
    b.build()


def same(got, want):
    return all(torch.equal(a, b) for a, b in zip(got, want))


def cuda(n, d, f, seed):
    return [t.cuda() for t in make(n, d, f, torch.bfloat16, seed)]


def test_capture_after_calls_on_another_stream():
    """The usual order of a program: calls on the current stream, a capture (on a
    stream of its own), calls on yet another stream, replays.  The captured
    calls do not wait for work outside the capture, and the later ones not for
    work that only the capture knows."""
    from gptq_qqq_calibration_gb300 import GatedFF
    sets = [cuda(100, 256, 512, 30 + k) for k in range(2)]
    op = GatedFF(256, 512, train_tokens=100)
    want = [op.backward(*s) for s in sets]
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        captured = op.backward(*sets[0])
    other = torch.cuda.Stream()
    got = op.backward(*sets[1], stream=other)
    torch.cuda.synchronize()
    assert same(got, want[1])
    for _ in range(2):
        for t in captured:
            t.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert same(captured, want[0])
    assert same(op.backward(*sets[1]), want[1])
    op.sync()


def test_two_streams_of_one_capture():
    """Calls on two streams of one capture use the workspace one after the other."""
    from gptq_qqq_calibration_gb300 import GatedFF
    n, d, f = 1500, 512, 1024
    sets = [cuda(n, d, f, 40 + k) for k in range(3)]
    op = GatedFF(d, f, train_tokens=n)
    want = [op.backward(*s) for s in sets]
    torch.cuda.synchronize()
    graph, side = torch.cuda.CUDAGraph(), torch.cuda.Stream()
    with torch.cuda.graph(graph):
        main = torch.cuda.current_stream()
        first = op.backward(*sets[0])
        side.wait_stream(main)
        with torch.cuda.stream(side):
            second = op.backward(*sets[1])
        third = op.backward(*sets[2])
        main.wait_stream(side)
    for _ in range(3):
        for t in (*first, *second, *third):
            t.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert same(first, want[0]) and same(second, want[1]) and same(third, want[2])
    op.sync()


def test_threads_default_streams():
    """Each thread's own default stream has the same handle value: calls of two
    threads follow one another all the same."""
    from gptq_qqq_calibration_gb300 import GatedFF, _lib
    n, d, f = 1500, 512, 1024
    lib, per_thread = _lib.load(), 2  # cudaStreamPerThread
    op = GatedFF(d, f, train_tokens=n)
    sets = [cuda(n, d, f, 60 + k) for k in range(2)]
    want = [op.backward(*s) for s in sets]
    got = [[tuple(torch.zeros_like(t) for t in w) for _ in range(20)] for w in want]
    torch.cuda.synchronize()
    status = [[], []]

    def work(k):
        ptrs = [t.data_ptr() for t in sets[k]]
        for out in got[k]:
            status[k].append(lib.gated_ff_backward(op.handle, ptrs[0], n, *ptrs[1:], *(t.data_ptr() for t in out),
                                                   per_thread))

    threads = [threading.Thread(target=work, args=(k,)) for k in range(2)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    assert status == [[_lib.HESS_OK] * 20] * 2
    assert all(same(out, want[k]) for k in range(2) for out in got[k])
    op.sync()


@pytest.mark.parametrize("limit", [0, 300, 1000, 3000])
def test_waits_that_run_out_end_the_kernel(limit):
    """Several tiles a pair of SMs, with a limit that some waits keep and others do
    not: the kernel ends, says so, and the handle works again."""
    from gptq_qqq_calibration_gb300 import GatedFF, HessError
    from gptq_qqq_calibration_gb300.gated_ff import gated_ff_set_timeout
    n, d, f = 2000, 256, 4096  # 256 tiles
    X, G, U, D = cuda(n, d, f, 70)
    op = GatedFF(d, f, train_tokens=n)
    want = (op.forward(X, G, U), *op.backward(X, G, U, D))
    op.sync()
    gated_ff_set_timeout(op.handle, limit)
    timeouts = 0
    for _ in range(10):
        op.forward(X, G, U), op.backward(X, G, U, D)
        try:
            op.sync()
        except HessError as e:
            assert "TIMEOUT" in str(e)
            timeouts += 1
    gated_ff_set_timeout(op.handle, 2_000_000_000)
    assert timeouts > 0 or limit > 0
    assert same((op.forward(X, G, U), *op.backward(X, G, U, D)), want)
    op.sync()


@pytest.mark.parametrize("limit", [0, 500, 2000, 8000])
def test_split_calls_on_another_stream_after_a_timeout(limit):
    """A call of split tiles that gave up leaves pieces that no tile was finished
    with.  Once it is reported, the next calls count from zero, on whatever
    stream they come."""
    from gptq_qqq_calibration_gb300 import GatedFF, HessError
    from gptq_qqq_calibration_gb300.gated_ff import gated_ff_set_timeout
    n, d, f = 300, 2568, 1096  # 18 tiles in 3 pieces each
    first, second = (cuda(n, d, f, 80 + k)[:3] for k in range(2))
    op = GatedFF(d, f)
    want = op.forward(*second)
    op.sync()
    streams = [torch.cuda.Stream() for _ in range(3)]
    torch.cuda.synchronize()
    for k in range(6):
        gated_ff_set_timeout(op.handle, limit)
        op.forward(*first, stream=streams[0])
        gated_ff_set_timeout(op.handle, 2_000_000_000)
        late = op.forward(*first, stream=streams[1])  # may run while the first is reported
        try:
            op.sync(streams[0])
        except HessError as e:
            assert "TIMEOUT" in str(e)
        got = [op.forward(*second, stream=streams[2]) for _ in range(3)]
        torch.cuda.synchronize()
        assert all(torch.equal(g, want) for g in got)
        del late
    op.sync()
