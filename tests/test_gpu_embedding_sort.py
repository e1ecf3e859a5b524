"""The embedding gradient's sort at sizes around 48 KB of shared memory, in a process
that has made no other call, and from threads whose calls need different amounts."""
import subprocess
import sys
import threading

import pytest
import torch

import sharded_optimizer_step_gb300 as ss

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


@pytest.fixture(scope="module", autouse=True)
def _built():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    ss.build()
    yield
    assert ss.device_status() == 0


def _gradient(n, vocab, seed):
    """Whole numbers, so that sums are exact: the gradient and what it has to be."""
    g = torch.Generator(device=DEV).manual_seed(seed)
    ids = torch.randint(0, vocab, (n,), generator=g, device=DEV)
    d = torch.randint(-8, 9, (n, 8), generator=g, device=DEV).float()
    want = torch.zeros(vocab, 8, device=DEV).index_add_(0, ids, d)
    return ss.embedding_grad(d, ids, torch.full((vocab, 8), 7.0, device=DEV)), want


FRESH = """
import sys
sys.path.insert(0, "tests")
import torch
from test_gpu_embedding_sort import _gradient
sms = torch.cuda.get_device_properties(0).multi_processor_count
for n in %s:
    got, want = _gradient(n, 331 * sms, n)       # 331 ids a block: 42368 bytes and 2 a token
    assert torch.equal(got, want), n
"""


@pytest.mark.parametrize("tokens", [(3326,), (3392,), (3325, 3328, 3360, 3391, 3393)])
def test_around_48_kb_in_a_fresh_process(tokens):
    done = subprocess.run([sys.executable, "-c", FRESH % (tokens,)], capture_output=True, text=True,
                          timeout=300)
    assert done.returncode == 0, done.stderr[-2000:]


def test_threads_with_large_and_small_sorts():
    failed = []

    def work(sizes):
        try:
            with torch.cuda.stream(torch.cuda.Stream(DEV)):
                for k in range(200):
                    got, want = _gradient(*sizes[k % len(sizes)], k)
                    if k % 20 == 0:
                        assert torch.equal(got, want), k
                torch.cuda.current_stream().synchronize()
        except Exception as e:  # told by the test
            failed.append(e)

    threads = [threading.Thread(target=work, args=(s,)) for s in
               ([(30000, 150_000)], [(12000, 150_000), (26000, 90_000)], [(5000, 100_000)])]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not failed, failed
