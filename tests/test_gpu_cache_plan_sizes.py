"""Plans of every number of requests, in a process that has planned nothing larger before, plans of different sizes
from host threads at once, and page numbers of every size."""
import os
import subprocess
import sys
import threading

import numpy as np
import pytest
import torch

from oracle import attention as oa

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(autouse=True, scope="module")
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA device")
    torch.cuda.init()


def i32(x):
    return torch.as_tensor(np.asarray(x), dtype=torch.int32, device="cuda")


def inputs(n):
    r = np.random.RandomState(n)
    lens, added = r.randint(0, 20, n), r.randint(0, 4, n)
    held = -(-lens // 16)
    table, at = np.full((n, 2), -1), 0
    for row, h in zip(table, held):
        row[:h] = np.arange(at, at + h)
        at += h
    return lens, added, table, np.arange(at, at + n), 16, int(added.sum()) + 3


def check(n):
    import linear_attention_sequence_rule_b200 as gdn
    lens, added, table, free, page, rows = inputs(n)
    t = i32(table)
    p = gdn.cache_plan(i32(lens), i32(added), t, i32(free), i32([0]), page, rows)
    want = oa.plan(lens, added, table, free, 0, page, rows)
    got = dict(p._asdict(), table=t)
    for name, w in want.items():
        assert np.array_equal(got[name].cpu().numpy().ravel(), np.asarray(w).ravel()), (n, name)


def test_sizes_near_the_shared_memory_that_needs_no_leave():
    sizes = [3969, 4010, 4011, 4050, 4051, 4052, 4053, 4090, 4094, 4095, 4096, 4097]
    code = f"from tests.test_gpu_cache_plan_sizes import check\nfor n in {sizes}: check(n)"
    r = subprocess.run([sys.executable, "-c", code], cwd=ROOT, capture_output=True, text=True, timeout=600)
    assert r.returncode == 0, r.stderr[-2000:]


def test_two_host_threads_plan_batches_of_different_sizes():
    import linear_attention_sequence_rule_b200 as gdn
    faults = []

    def loop(n):
        try:
            lens, added, table, free, page, rows = inputs(n)
            dev = [i32(x) for x in (lens, added, table, free, [0])]
            want = oa.plan(lens, added, table, free, 0, page, rows)["slots"]
            stream = torch.cuda.Stream()
            torch.cuda.synchronize()
            got = [gdn.cache_plan(*dev, page, rows, stream=stream).slots for _ in range(100)]
            stream.synchronize()
            assert all(g.tolist() == want for g in got[::33])
        except Exception as e:  # noqa: BLE001 (reported by the test)
            faults.append((n, repr(e)))

    threads = [threading.Thread(target=loop, args=(n,)) for n in (16384, 4200, 5000)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not faults, faults


@pytest.mark.parametrize("page", [16, 32, 64, 128])
def test_page_numbers_that_no_slot_holds(page):
    """A slot is page number x page + offset, or -1 where 32 bits do not hold it: never a slot of another page."""
    import linear_attention_sequence_rule_b200 as gdn
    top = 2 ** 31 // page
    numbers = [0, 5, -1, -2, top - 1, top, top + 3, 2 * top, 2 * top + 1, 2 ** 31 - 1, -top, -top - 1, -2 * top, -2 ** 31]
    n = len(numbers)
    t = i32([[x, -1] for x in numbers])  # every request holds three tokens and fills its page, then takes one
    p = gdn.cache_plan(i32([3] * n), i32([page - 2] * n), t, i32(numbers), i32([0]), page, n * (page - 2))
    assert p.status.tolist() == [0, 0]
    want = []
    for x in numbers:
        slots = [x * page + j for j in range(3, page)] + [x * page]
        want += [s if -2 ** 31 <= s < 2 ** 31 else -1 for s in slots]
    assert p.slots.tolist() == want and t[:, 1].tolist() == numbers
    assert p.positions.tolist() == list(range(3, page + 1)) * n
