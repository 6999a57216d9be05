"""The device status words, read and cleared in one go."""
import statistics
import threading
import time

import pytest
import torch

from fp8_moe_routed_gb300 import binding as fb

pytestmark = pytest.mark.gpu


def bad_ids():
    """A sort with an id past the experts: BAD_EXPERT in one unit's word."""
    fb.sort_tokens(torch.tensor([[9]], dtype=torch.int32, device="cuda"), 4)


def too_many_rows():
    """A quantisation whose sizes add up past the buffer: GROUPS_EXCEED_M in another's."""
    fb.mxfp4_quantize_rows(torch.zeros(4, 32, dtype=torch.bfloat16, device="cuda"),
                           torch.tensor([5], dtype=torch.int32, device="cuda"))


def negative_group():
    """NEGATIVE_GROUP in a third one's."""
    fb.quantize_rows(torch.zeros(4, 32, dtype=torch.bfloat16, device="cuda"),
                     torch.tensor([-1], dtype=torch.int32, device="cuda"))


def test_bits_of_all_units_together_and_once():
    fb.read_status()
    bad_ids()
    too_many_rows()
    negative_group()
    assert fb.read_status() == (fb.STATUS_BAD_EXPERT | fb.STATUS_GROUPS_EXCEED_M |
                                fb.STATUS_NEGATIVE_GROUP)
    assert fb.read_status() == 0
    fb.selftest_wait_timeout(1)
    assert fb.read_status() & fb.STATUS_WAIT_TIMEOUT
    assert fb.read_status() == 0


def test_every_bit_reaches_one_reader():
    """Threads that set a bit and read on streams of their own: each bit is seen by some
    reading, by the setter's own or by one that came before it, and none is left behind."""
    fb.read_status()
    rounds, seen, lock = 200, [0], threading.Lock()
    start = threading.Barrier(3)

    def reader(stop):
        stream = torch.cuda.Stream()
        start.wait()
        with torch.cuda.stream(stream):
            while not stop.is_set():
                got = fb.read_status()
                if got:
                    with lock:
                        seen[0] += 1

    stop = threading.Event()
    threads = [threading.Thread(target=reader, args=(stop,)) for _ in range(2)]
    for t in threads:
        t.start()
    start.wait()
    stream = torch.cuda.Stream()
    missed = 0
    with torch.cuda.stream(stream):
        for _ in range(rounds):
            with lock:
                before = seen[0]
            bad_ids()
            stream.synchronize()
            own = fb.read_status()
            # the readers' counts are taken under their lock after their reading has returned
            limit = time.perf_counter() + 2.0
            while not own and time.perf_counter() < limit:
                with lock:
                    if seen[0] > before:
                        break
            else:
                missed += not own
    stop.set()
    for t in threads:
        t.join()
    assert missed == 0
    assert fb.read_status() == 0


def test_cost():
    """One launch, one copy and one wait: a few times the cost of reading a value back, not
    that of a copy and two waits for every kernel file (which was fifteen times it)."""
    x = torch.ones(1, device="cuda")

    def median(f):
        times = []
        for _ in range(200):
            t = time.perf_counter()
            f()
            times.append(time.perf_counter() - t)
        return statistics.median(times)

    for f in (fb.read_status, x.item):
        median(f)
    assert median(fb.read_status) <= 6 * median(x.item)
