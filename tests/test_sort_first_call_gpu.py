"""sort_by_expert() as the first call of a process, and from several threads: the shared memory that a
launch may use is set per kernel and outlives the call, so an order that is made after a larger one
says nothing about its own setting.  The sizes lie on both sides of those at which the tables and the
kernel's static shared memory together pass 48 KB."""

import os
import subprocess
import sys

import pytest

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

ONE = """
import sys
import torch
import moe_grouped_matrix_gb300 as G
import moe_reference as R
slots, experts = int(sys.argv[1]), int(sys.argv[2])
e = torch.randint(0, experts, (slots, 1), generator=torch.Generator().manual_seed(slots)).to(torch.int32)
order = G.sort_by_expert(e.cuda(), experts)
sizes, rows, source = R.order_of(e.numpy(), experts)
assert order.group_sizes.tolist() == sizes.tolist()
assert order.rows.tolist() == rows.tolist() and order.source.tolist() == source.tolist()
"""

MANY = """
import threading
import torch
import moe_grouped_matrix_gb300 as G
wrong = []
choices = {n: torch.randint(0, n, (3000, 2), dtype=torch.int32).cuda() for n in (264, 360, 1024)}
want = {n: G.sort_by_expert(e, n) for n, e in choices.items()}
torch.cuda.synchronize()

def sort(n):
    stream = torch.cuda.Stream()
    try:
        for _ in range(400):
            got = G.sort_by_expert(choices[n], n, stream=stream)
        stream.synchronize()
        if not all(torch.equal(a, b) for a, b in zip(got, want[n])):
            wrong.append(n)
    except Exception as e:
        wrong.append((n, str(e)))

threads = [threading.Thread(target=sort, args=(n,)) for n in choices for _ in range(2)]
for t in threads:
    t.start()
for t in threads:
    t.join()
assert not wrong, wrong
"""


def run(code, *args):
    env = dict(os.environ, PYTHONPATH=os.pathsep.join((ROOT, os.path.join(ROOT, "tests"))))
    got = subprocess.run([sys.executable, "-c", code, *map(str, args)], cwd=ROOT, env=env, capture_output=True,
                         text=True, timeout=300)
    assert got.returncode == 0, got.stderr[-2000:]


@pytest.mark.parametrize("slots,experts", [(2048, 359), (2048, 360), (2048, 361), (4096, 297), (4096, 298),
                                           (4096, 299), (16384, 250), (256, 1024)])
def test_the_first_call_of_a_process(slots, experts):
    run(ONE, slots, experts)


def test_threads_with_different_numbers_of_experts():
    run(MANY)
