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


def test_arguments_that_are_not_tensors():
    x, off = rand((4, 8), BF, 1).to(DEV), offsets_of([4]).to(DEV)
    w, t = torch.zeros(1, 8, 8, device=DEV), torch.zeros(4, dtype=torch.int64, device=DEV)
    for call in (lambda: mf.grouped_linear_wgrad(x, x, off, w, workspace=[1]),
                 lambda: mf.grouped_linear_wgrad_ckpt(x, *mf.ckpt_quantize(x), off, w, workspace=[1]),
                 lambda: mf.embedding_grad(x, t, w[0], workspace=256), lambda: mf.embedding(w[0], t, out=[1.0]),
                 lambda: mf.embedding(w[0], t, dtype=BF, out=[1.0]), lambda: mf.embedding(w[0], [0, 1]),
                 lambda: mf.grouped_linear(x, [1], off), lambda: mf.grouped_linear(x, w.to(BF), off, out=3),
                 lambda: mf.grouped_linear_wgrad(x, None, off, w), lambda: mf.ckpt_restore(3, None),
                 lambda: mf.ckpt_restore(mf.ckpt_quantize(x)[0], None), lambda: mf.ckpt_quantize(x, codes=1)):
        with pytest.raises(TypeError, match="must be a tensor"):
            call()


def test_lookups_beyond_one_launch():
    # 257 bf16 columns take two workgroups a token: 2^23 tokens are as many as
    # one launch has
    n, vocab, d = (1 << 23) + 11, 1000, 257
    table = rand((vocab, d), BF, 1).to(DEV)
    t = torch.randint(0, vocab, (n,), generator=torch.Generator().manual_seed(2), dtype=torch.int32).to(DEV)
    t[5], t[-2] = -1, vocab
    out = mf.embedding(table, t, out=torch.full((n, d), 7.0, dtype=BF, device=DEV))
    assert not out[5].any() and not out[-2].any()
    for lo in range(0, n, 1 << 21):
        part = t[lo:lo + (1 << 21)].long()
        on = (part >= 0) & (part < vocab)
        assert torch.equal(out[lo:lo + (1 << 21)], torch.where(on[:, None], table[part.clamp(0, vocab - 1)], 0))


@pytest.mark.parametrize("d", [2, 4])
@pytest.mark.parametrize("beta", [0.0, 1.0])
def test_table_gradients_beyond_one_launch(d, beta):
    # a workgroup takes four table rows: 2^26 rows are as many as one launch has
    vocab, n = (1 << 26) + 5, 3000
    g = torch.Generator().manual_seed(3)
    t = torch.randint(0, vocab, (n,), generator=g)
    t[:400] = torch.arange(400) % 18 + vocab - 18                      # both sides of the launches' border,
    t[400:600] = vocab - 1                                             # one of them often
    t[600], t[601], t[602] = 0, -1, vocab
    dy = rand((n, d), F32, 4)
    old = 0.5 if beta else 0.0
    grad = mf.embedding_grad(dy.to(DEV), t.to(DEV), torch.full((vocab, d), 0.5 if beta else float("nan"), device=DEV), beta=beta)
    on = (t >= 0) & (t < vocab)
    rows, place = torch.unique(t[on], return_inverse=True)
    compact = torch.full((n,), -1)
    compact[on] = place
    want, mag, terms = ref.embedding_grad(dy, compact, rows.numel(), 1.0)
    assert ref.worst(grad[rows.to(DEV)], want + old, (terms[:, None] + 2) * ref.U * mag + 2 * ref.U * old) <= 1.0
    grad[rows.to(DEV)] = old
    assert (grad == old).all()          # every other row


def test_checkpoints_beyond_one_launch():
    # 32 blocks a workgroup: 2^29 rows of one block are as many as one launch
    # has.  The parts of a long activation have the checkpoints that they have
    # alone.
    rows = (1 << 29) + 33
    x = torch.empty(rows, 1, dtype=BF, device=DEV).normal_(generator=torch.Generator(DEV).manual_seed(1))
    codes, scales = mf.ckpt_quantize(x)
    back = mf.ckpt_restore(codes, scales, out=torch.full((rows, 1), 7.0, dtype=BF, device=DEV))
    for lo in range(0, rows, 1 << 28):
        c, s = mf.ckpt_quantize(x[lo:lo + (1 << 28)])
        assert torch.equal(codes[lo:lo + (1 << 28)], c) and torch.equal(scales[lo:lo + (1 << 28)], s)
        assert torch.equal(back[lo:lo + (1 << 28)], mf.ckpt_restore(c, s))
    cr, sr = ref.ckpt_quantize(x[-100:])
    assert torch.equal(codes[-100:].cpu(), torch.from_numpy(cr)) and torch.equal(scales[-100:].cpu(), torch.from_numpy(sr))


def test_large_output_projection():
    # 34 GB of outputs: more than 2^23 tiles of 32 x 64, 2^18 of those that run
    rows, n, k = 131072, 131200, 64
    x, w = rand((rows, k), BF, 1).to(DEV), rand((1, n, k), BF, 2, 0.05).to(DEV)
    off = torch.tensor([0, rows], dtype=torch.int32, device=DEV)
    y = mf.grouped_linear(x, w, off)
    wd = w[0].double().t().contiguous()
    for lo in (0, 65536 - 128, rows - 256):
        a = x[lo:lo + 256].double()
        want, mag = a @ wd, a.abs() @ wd.abs()
        assert float(((y[lo:lo + 256].double() - want).abs() / (ref.half_step(BF) * want.abs() + k * ref.U * mag)).max()) <= 1.0


def test_timing_leaves_captured_launches_alone():
    x, w, off = rand((10, 16), BF, 1).to(DEV), rand((2, 8, 16), BF, 2).to(DEV), offsets_of([4, 6]).to(DEV)
    want = mf.grouped_linear(x, w, off)
    y = torch.zeros_like(want)
    mf.timing.enable(True)
    try:
        mf.timing.reset()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            mf.grouped_linear(x, w, off, out=y)
        for _ in range(3):
            y.zero_()
            graph.replay()
            assert torch.equal(y, want)
        assert mf.timing.read("grouped")[1] == 0
        mf.grouped_linear(x, w, off)
        assert mf.timing.read("grouped")[1] == 1
    finally:
        mf.timing.enable(False)
        mf.timing.reset()
