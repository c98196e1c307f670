"""Ways of calling the gradient operators on the GPU: host threads on one
stream, captured steps beside them.
"""

import threading

import pytest
import torch

import grads_ref as ref
import matrix_optimizer_step_owner_amd as mf
from test_gpu_grads import BF, DEV, F32, _need_gpu, offsets_of, rand, tokens_of  # noqa: F401

pytestmark = pytest.mark.gpu


def test_host_threads_on_one_stream():
    # each thread's calls give what they give alone, whatever the other enqueues
    # between their launches (several sort passes; parts and their sum)
    stream = torch.cuda.Stream()
    states, want = [], []
    for i, (n, vocab, d) in enumerate([(9001, 70000, 24), (20000, 5000, 40)]):
        counts = [[9001], [5000, 15000]][i]
        states.append({"dy": rand((n, d), BF, i).to(DEV), "t": tokens_of("zipf", n, vocab, i).to(DEV), "vocab": vocab, "d": d,
                       "x": rand((n, 64), BF, 5 + i).to(DEV), "off": offsets_of(counts).to(DEV), "e": len(counts)})

    def both(s):
        g = mf.embedding_grad(s["dy"], s["t"], torch.empty(s["vocab"], s["d"], device=DEV))
        w = mf.grouped_linear_wgrad(s["dy"], s["x"], s["off"], torch.empty(s["e"], s["d"], 64, device=DEV))
        return g, w

    for s in states:
        want.append(both(s))
    torch.cuda.synchronize()
    got, errors = [[], []], []
    start = threading.Barrier(2)

    def work(i):
        try:
            with torch.cuda.stream(stream):
                start.wait(30)
                for _ in range(8):
                    got[i].append(both(states[i]))
        except Exception as e:      # reported below, by the test's own thread
            errors.append(e)

    threads = [threading.Thread(target=work, args=(i,)) for i in range(2)]
    for t in threads:
        t.start()
    for t in threads:
        t.join(60)
    torch.cuda.synchronize()
    assert not errors and [len(g) for g in got] == [8, 8]
    for i in range(2):
        for g, w in got[i]:
            assert torch.equal(g, want[i][0]) and torch.equal(w, want[i][1])
