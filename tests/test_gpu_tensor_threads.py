"""One list of tensors used by several host threads on one stream."""
import math
import threading

import numpy as np
import pytest
import torch

from gpu_common import need_gpu, say

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("chunks", [3, 700, 5000])
def test_threads_on_one_stream(chunks):
    """Sums of squares and largest magnitudes at once: every result equals the
    one of a thread alone, to the bit."""
    gns = need_gpu()
    rng = np.random.default_rng(90)
    grads = torch.from_numpy(rng.normal(size=(chunks, 5))).float().cuda()
    lst = gns.tensor_list(list(grads))
    assert lst.info.chunks == chunks
    want = {o: gns.grad_norm(lst, ord=o, max_norm=1.0, per_tensor=True) for o in (2, math.inf)}
    torch.cuda.synchronize()
    got, failed = [], []
    start = threading.Barrier(4)

    def worker(ord):
        try:
            start.wait()
            got.extend([(ord, gns.grad_norm(lst, ord=ord, max_norm=1.0, per_tensor=True)) for _ in range(50)])
        except Exception as e:  # noqa: BLE001 (reported below)
            failed.append(e)

    say("threads on one stream", chunks)
    threads = [threading.Thread(target=worker, args=(o,)) for o in (2, math.inf, 2, math.inf)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    assert not failed and len(got) == 200
    for ord, g in got:
        assert torch.equal(g.result, want[ord].result) and torch.equal(g.tensor_norms, want[ord].tensor_norms)
