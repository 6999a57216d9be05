"""Calls of one kernel at sizes that need different amounts of shared memory, in turn: a
captured graph and a second thread must not see the limits of another call."""
import threading

import pytest
import torch

from fp8_moe_routed_gb300 import binding as fb

pytestmark = pytest.mark.gpu

BF16 = torch.bfloat16


def norms(T, H, seed):
    """Inputs, and a call that runs both directions on them."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    x, y, dr, dh = (torch.randn(T, H, generator=g, device="cuda").to(BF16) for _ in range(4))
    w = 1 + 0.1 * torch.randn(H, generator=g, device="cuda")

    def run():
        r, h, rp, rq = fb.norm_fwd(x, y, w, w, gate=w, gate_kind="channel")
        return (r, h) + fb.norm_bwd(dr, dh, r, y, w, w, rp, rq, gate=w, gate_kind="channel")
    return run


def sorts(T, k, E, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    ids = torch.randint(0, E, (T, k), generator=g, device="cuda", dtype=torch.int32)
    return lambda: fb.sort_tokens(ids, E)


# a large call and a small one of the same kernel
PAIRS = {
    "norms": (lambda: norms(300, 8192, 1), lambda: norms(1, 8192, 2), lambda: norms(5, 512, 3)),
    "sort": (lambda: sorts(3000, 4, 1024, 4), lambda: sorts(300, 8, 2, 5),
             lambda: sorts(3000, 4, 8, 6)),
}


@pytest.mark.parametrize("what", sorted(PAIRS))
def test_a_graph_keeps_its_limits(what):
    large, *small = (make() for make in PAIRS[what])
    want = [t.clone() for t in large()]
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = large()
    for t in got:
        t.zero_()
    for run in small:
        run()
    graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    assert fb.read_status() == 0


@pytest.mark.parametrize("what", sorted(PAIRS))
def test_threads_with_streams_of_their_own(what):
    calls = [make() for make in PAIRS[what]]
    want = [[t.clone() for t in run()] for run in calls]
    torch.cuda.synchronize()
    faults = []

    def work(run, expected):
        try:
            stream = torch.cuda.Stream()
            with torch.cuda.stream(stream):
                for _ in range(100):
                    got = run()
                    if not all(torch.equal(a, b) for a, b in zip(got, expected)):
                        faults.append("other results")
                        return
        except Exception as e:  # noqa: BLE001 -- reported by the assertion below
            faults.append(repr(e))

    threads = [threading.Thread(target=work, args=a) for a in zip(calls, want)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert faults == []
    assert fb.read_status() == 0
