"""Ways of calling routing, the exchange of rows, layer norm and the 8-bit float
products on the GPU: every tile kernel, streams, host threads, graphs, buffers
past 4 GiB, workspaces, arguments, and a whole training step of them with the Muon
step and the AdamW tail.
"""

import ctypes
import threading

import pytest
import torch

import grads_ref as gref
import layers_ref as ref
import matrix_optimizer_step_owner_amd as mf
from matrix_optimizer_step_owner_amd import _lib
from test_gpu_grads import BF, DEV, F32, NAN, _need_gpu, offsets_of, rand  # noqa: F401
from test_gpu_layers import activations, logits_of, plan_of

pytestmark = pytest.mark.gpu


# ---------------------------------------------------------------------------
# Each kernel of the 8-bit products, on ragged segments and widths
# ---------------------------------------------------------------------------
# kernel (rows, columns of its tile): rows of each expert, n, k
TILES = [((32, 32), [3, 0, 30, 1], 100, 1000), ((32, 32), [33, 31], 513, 136), ((32, 64), [70, 0, 200, 9], 1000, 384), ((32, 64), [4] * 100, 1100, 200),
         ((32, 64), [16, 17, 0, 18], 14336, 4100), ((128, 128), [130, 0, 300, 127, 129, 1], 2999, 264), ((128, 128), [40] * 60, 1100, 128),
         ((128, 128), [1000, 24, 2000, 900], 1025, 640), ((256, 256), [2100, 0, 255, 257, 3000, 513], 3900, 200), ((256, 256), [9000], 4100, 384),
         ((256, 256), [700, 1500, 300, 511, 2300, 2049], 2048, 256)]


@pytest.mark.parametrize("shape,counts,n,k", TILES)
def test_every_tile(shape, counts, n, k):
    rows = sum(counts)
    t = _lib.MfsdpGroupedTile()
    _lib.check(_lib.load().mfsdp_scaled_linear_tile(len(counts), rows, n, k, ctypes.byref(t)))
    assert (t.rows, t.cols) == shape
    off = offsets_of(counts)
    x, w = rand((rows, k), BF, 1).to(DEV), rand((len(counts), n, k), BF, 2, 0.05).to(DEV)
    q, qw = mf.scaled_quantize(x), mf.scaled_quantize_weight(w)
    out = torch.full((rows, n + 24), 7.0, dtype=BF, device=DEV)
    y = mf.scaled_linear(*q, *qw, off.to(DEV), out=out[:, 8:8 + n])
    power = lambda s: torch.exp2(s.double() - 127)
    xv = q[0].double() * power(q[1]).repeat_interleave(128, 1)
    for e, (lo, hi) in enumerate(gref.segments(off, rows)):
        if hi == lo:
            continue
        wv = qw[0][e].double() * power(qw[1][e]).repeat_interleave(128, 0)[:n].repeat_interleave(128, 1)
        want, mag = xv[lo:hi] @ wv.t(), xv[lo:hi].abs() @ wv.t().abs()
        # the sum of the eights' largest is under the sum of all magnitudes
        bound = ref.half_step(BF) * want.abs() + (1 + 2 ** -8) * (2 ** -10 + (k + 8) * ref.U) * mag + 1e-38
        assert float(((y[lo:hi].double() - want).abs() / bound).max()) <= 1.0
        # and typically far nearer: the sums' own error is 5e-5 of the result at most
        assert float((y[lo:hi].double() - want).norm() / want.norm()) <= 2 ** -9 + 1e-4
    assert (out[:, :8] == 7).all() and (out[:, 8 + n:] == 7).all()


@pytest.mark.parametrize("experts", [63, 65, 300, 5000, 9000])
def test_tiles_of_many_experts(experts):
    # most of them without a row, some with several tiles
    n, k = 40, 128
    c = torch.where(torch.rand(experts, generator=torch.Generator().manual_seed(experts)) < 0.2, 3000 // experts + 1, 0)
    c[0], c[experts // 2], c[-1] = 700, 130, 65
    c = c.tolist()
    rows = sum(c)
    x, w = rand((rows, k), BF, 1).to(DEV), rand((experts, n, k), BF, 2, 0.05).to(DEV)
    q, qw = mf.scaled_quantize(x), mf.scaled_quantize_weight(w)
    y = mf.scaled_linear(*q, *qw, offsets_of(c).to(DEV))
    e = torch.repeat_interleave(torch.arange(experts), torch.tensor(c)).to(DEV)
    power = lambda s: torch.exp2(s.double() - 127)
    xv = q[0].double() * power(q[1])
    wv = (qw[0].double() * power(qw[1]).repeat_interleave(128, 1)[:, :n])[e]
    want, mag = (wv * xv[:, None]).sum(2), (wv * xv[:, None]).abs().sum(2)
    bound = ref.half_step(BF) * want.abs() + (1 + 2 ** -8) * (2 ** -10 + (k + 8) * ref.U) * mag + 1e-38
    assert float(((y.double() - want).abs() / bound).max()) <= 1.0


def test_wrong_offsets_stay_inside():
    # offsets that decrease or lie outside give wrong results, and touch nothing else
    x, w = rand((300, 256), BF, 1).to(DEV), rand((3, 200, 256), BF, 2, 0.05).to(DEV)
    q, qw = mf.scaled_quantize(x), mf.scaled_quantize_weight(w)
    for off in ([0, 400, 100, 300], [-50, 20, 1000, 2 ** 31 - 1], [300, 200, 100, 0], [5, 5, 5, 5]):
        wide = torch.full((310, 200), 7.0, dtype=BF, device=DEV)
        mf.scaled_linear(*q, *qw, torch.tensor(off, dtype=torch.int32, device=DEV), out=wide[:300])
        assert (wide[300:] == 7).all()


# ---------------------------------------------------------------------------
# A step of all of them
# ---------------------------------------------------------------------------
def state_of(seed, tokens=200, d=96, n=64, experts=16, k=4, dtype=BF):
    s = {"x": activations(tokens, d, dtype, seed), "gain": 1 + rand((d,), F32, seed + 1, 0.1), "shift": rand((d,), F32, seed + 2, 0.1),
         "wr": rand((1, experts, d), dtype, seed + 3, 0.2), "bias": rand((experts,), F32, seed + 4, 0.02), "w": rand((experts, n, d), dtype, seed + 5, 0.1),
         "v": rand((experts, d, n), dtype, seed + 6, 0.1), "dy": rand((tokens, d), dtype, seed + 7),
         "mask": torch.rand(tokens, generator=torch.Generator().manual_seed(seed)) < 0.9, "one": torch.tensor([0, tokens], dtype=torch.int32)}
    s = {key: t.to(DEV) for key, t in s.items()}
    for key in ("gain", "shift", "wr", "w", "v"):
        s["d" + key] = torch.zeros_like(s[key], dtype=F32)
    return dict(s, k=k, eight=dtype == BF)


def forward(s):
    s["h"] = mf.layer_norm(s["x"], s["gain"], s["shift"])
    s["logits"] = mf.grouped_linear(s["h"], s["wr"], s["one"])
    s["experts"], s["weights"] = mf.route(s["logits"], s["k"], scores="sigmoid", bias=s["bias"], groups=4, top_groups=2, scale=1.5, mask=s["mask"])
    s["plan"] = mf.route_plan(s["experts"], s["w"].shape[0])
    rows = s["x"].shape[0] * s["k"]
    s["xs"] = mf.route_dispatch(s["h"], s["plan"].place, out=torch.zeros(rows, s["x"].shape[1], dtype=s["x"].dtype, device=DEV))
    s["a"] = mf.grouped_linear(s["xs"], s["w"], s["plan"].offsets, out=torch.zeros(rows, s["w"].shape[1], dtype=s["x"].dtype, device=DEV))
    s["b"] = s["a"] * s["a"]
    s["o"] = mf.grouped_linear(s["b"], s["v"], s["plan"].offsets, out=torch.zeros_like(s["xs"]))
    s["y"] = mf.route_combine(s["o"], s["plan"].place, s["weights"])
    return s["y"]


def backward(s):
    off = s["plan"].offsets
    do, s["dweights"] = mf.route_combine_grad(s["dy"], s["o"], s["plan"].place, s["weights"], dh=torch.zeros_like(s["o"]))
    mf.grouped_linear_wgrad(do, s["b"], off, s["dv"])
    db = mf.grouped_linear_dgrad(do, s["v"], off, out=torch.zeros_like(s["b"]))
    da = 2 * s["a"] * db
    mf.grouped_linear_wgrad(da, s["xs"], off, s["dw"])
    dxs = mf.grouped_linear_dgrad(da, s["w"], off, out=torch.zeros_like(s["xs"]))
    s["dlogits"] = mf.route_grad(s["dweights"], s["logits"], s["experts"], scores="sigmoid", scale=1.5)
    mf.grouped_linear_wgrad(s["dlogits"], s["h"], s["one"], s["dwr"])
    dh = mf.grouped_linear_dgrad(s["dlogits"], s["wr"], s["one"])
    mf.route_combine(dxs, s["plan"].place, beta=1.0, out=dh)
    s["dh"] = dh.clone()
    s["dx"] = mf.layer_norm_grad(dh, s["x"], s["gain"], s["dgain"], s["dshift"])
    if s["eight"]:      # the same products from 8-bit copies
        c = mf.scaled_quantize_weight(s["w"], both=True)
        s["a8"] = mf.scaled_linear(*mf.scaled_quantize(s["xs"]), *c[:2], off, out=torch.zeros_like(s["a"]))
        s["dxs8"] = mf.scaled_linear(*mf.scaled_quantize(da), *c[2:], off, out=torch.zeros_like(s["xs"]))
    mf.route_balance(s["bias"], off.diff(), 1e-3)


RESULTS = ("y", "experts", "weights", "dx", "dgain", "dshift", "dwr", "dw", "dv", "dlogits", "bias")


def step(s):
    forward(s)
    backward(s)
    got = [s[key].clone() for key in RESULTS] + [s["plan"].offsets.clone(), s["plan"].place.clone()]
    return got + ([s["a8"].clone(), s["dxs8"].clone()] if s["eight"] else [])


def test_training_step_against_autograd():
    # fp32: the whole step's gradients against 64-bit automatic differentiation at
    # the same choice of experts.  Each operator is off by at most 130 terms of U
    # of its operands' sizes (sums over 96 columns, 64, 4 and 200 rows), eleven
    # of them in a chain: 11 * 130 * U = 1.7e-4 of the sizes that a gradient adds
    # up, which here are under ten times the gradient.
    s = state_of(1, dtype=F32)
    step(s)
    leaf = {key: s[key].detach().cpu().double().requires_grad_() for key in ("x", "gain", "shift", "wr", "w", "v")}
    xc = leaf["x"] - leaf["x"].mean(1, keepdim=True)
    h = xc / torch.sqrt((xc * xc).mean(1, keepdim=True) + 1e-5) * leaf["gain"] + leaf["shift"]
    p = torch.sigmoid(h @ leaf["wr"][0].t())
    e = s["experts"].cpu().long()
    on = e >= 0
    assert torch.equal(on.all(1), s["mask"].cpu()) and torch.equal(on.any(1), s["mask"].cpu())
    sel = torch.where(on, p.gather(1, e.clamp(min=0)), 0.0)
    wts = 1.5 * sel / (sel.sum(1, keepdim=True) + 1e-20)
    a = torch.einsum("tjnd,td->tjn", leaf["w"][e.clamp(min=0)], h)
    o = torch.einsum("tjdn,tjn->tjd", leaf["v"][e.clamp(min=0)], a * a)
    y = (wts[:, :, None] * torch.where(on[:, :, None], o, 0.0)).sum(1)
    y.backward(s["dy"].cpu().double())
    assert float((s["y"].cpu().double() - y.detach()).norm() / y.detach().norm()) <= 1.7e-3
    for key in leaf:
        want = leaf[key].grad
        assert float((s["d" + key].cpu().double() - want).norm() / want.norm()) <= 1.7e-3, key


def test_eight_bit_products_are_near():
    # e4m3 has half steps of 2^-4 relative at most, typically a third of that, on both
    # operands: 2^-4 sqrt(2) / sqrt(3) = 5% of a sum of random terms, 8% as a bar
    s = state_of(2)
    step(s)
    for eight, whole in (("a8", "a"),):
        assert float((s[eight].float() - s[whole].float()).norm() / s[whole].float().norm()) <= 0.08


def test_together_with_the_step():
    # gradients where the two optimizers take them: experts' and the router's
    # matrices in a Muon step, gain and shift in the packed AdamW tail
    s = state_of(3)
    packed, at = mf.tail_pack([s["gain"], s["shift"]])
    gpacked = torch.full_like(packed, NAN)
    d = s["gain"].numel()
    for i, key in enumerate(("gain", "shift")):
        s[key], s["d" + key] = packed[at[i]:at[i] + d], gpacked[at[i]:at[i] + d]
    for key in ("w", "v", "wr"):
        s["d" + key] = torch.zeros_like(s[key])
    step(s)
    # each gradient against the formula, from what the call before it gave
    (dx, bx), (dw, bw), (db, bb) = ref.norm_grad(s["dh"], s["x"], s["gain"], 1e-5, True)
    assert gref.worst(s["dx"], dx, bx + ref.half_step(BF) * dx.abs()) <= 1.0
    assert gref.worst(s["dgain"], dw, bw + ref.U * dw.abs()) <= 1.0 and gref.worst(s["dshift"], db, bb + ref.U * db.abs()) <= 1.0
    want, bound = ref.route_grad(s["dweights"], s["logits"], s["experts"], "sigmoid", True, 1.5)
    assert gref.worst(s["dlogits"], want, bound + ref.half_step(BF) * want.abs()) <= 1.0
    before = {key: s[key].clone() for key in ("w", "v", "wr", "gain", "shift")}
    W = [m for key in ("w", "v", "wr") for m in s[key]]
    G = [m for key in ("dw", "dv", "dwr") for m in s[key]]
    mf.MuonStep(W, G, [torch.zeros_like(m) for m in W]).step(lr=0.02)
    gpacked = torch.nan_to_num(gpacked)     # between the segments
    mf.adamw_tail(packed, gpacked, torch.zeros_like(packed), torch.zeros_like(packed), lr=0.01, beta1=0.9, beta2=0.95, eps=1e-8, weight_decay=0.01, step=1)
    for key, old in before.items():
        assert torch.isfinite(s[key]).all() and not torch.equal(s[key], old), key


def test_graph_replays_follow_the_inputs():
    s, s2 = state_of(1), state_of(2, tokens=1500)
    step(s), step(s2)                       # loads the kernels
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph, second = torch.cuda.CUDAGraph(), torch.cuda.CUDAGraph()
    with torch.cuda.stream(side):
        with torch.cuda.graph(graph, stream=side):
            got = step(s)
        with torch.cuda.graph(second, stream=side):     # a second graph beside it
            got2 = step(s2)
    torch.cuda.synchronize()
    for i in range(4):
        new, new2 = state_of(20 + i), state_of(30 + i, tokens=1500)
        for a, b in ((s, new), (s2, new2)):
            for key in ("x", "gain", "shift", "wr", "bias", "w", "v", "dy", "mask"):
                a[key].copy_(b[key])
        graph.replay()
        second.replay()
        torch.cuda.synchronize()
        for a, b in ((got, new), (got2, new2)):
            for g, want in zip(a, step(b)):
                assert torch.equal(g, want), i


def test_side_streams_and_threads():
    # two streams at once, and two host threads on one stream, each with its own
    # workspace, give what one gives
    states = [state_of(5, tokens=3000), state_of(6, tokens=2500)]

    def fresh(i):
        return {key: t.clone() if torch.is_tensor(t) else t for key, t in states[i].items()}

    want = [step(fresh(i)) for i in range(2)]
    torch.cuda.synchronize()
    streams, got = [torch.cuda.Stream(), torch.cuda.Stream()], [None, None]
    copies = [fresh(0), fresh(1)]
    torch.cuda.synchronize()
    for i in range(2):
        with torch.cuda.stream(streams[i]):
            got[i] = step(copies[i])
    torch.cuda.synchronize()
    for i in range(2):
        assert all(torch.equal(a, b) for a, b in zip(got[i], want[i]))
    runs, errors = [[], []], []
    stream, start = torch.cuda.Stream(), threading.Barrier(2)
    inputs = [[fresh(i) for _ in range(3)] for i in range(2)]
    torch.cuda.synchronize()

    def work(i):
        try:
            with torch.cuda.stream(stream):
                start.wait(30)
                for s in inputs[i]:
                    runs[i].append(step(s))
        except Exception as e:      # reported below, by the test's own thread
            errors.append(e)

    threads = [threading.Thread(target=work, args=(i,)) for i in range(2)]
    for t in threads:
        t.start()
    for t in threads:
        t.join(60)
    torch.cuda.synchronize()
    assert not errors and [len(r) for r in runs] == [3, 3]
    for i in range(2):
        for r in runs[i]:
            assert all(torch.equal(a, b) for a, b in zip(r, want[i]))


def test_given_workspaces():
    e = plan_of(3000, 4, 16, 1)         # any list of numbers will do as experts
    x, dy, w = activations(500, 300, F32, 1).to(DEV), rand((500, 300), F32, 2).to(DEV), rand((300,), F32, 3).to(DEV)
    ws = torch.empty(1 << 24, dtype=torch.uint8, device=DEV)
    a, b = mf.route_plan(e.to(DEV), 900, workspace=ws), mf.route_plan(e.to(DEV), 900)
    assert torch.equal(a.offsets, b.offsets) and torch.equal(a.place, b.place)
    g = [torch.zeros(300, device=DEV) for _ in range(2)]
    assert torch.equal(mf.layer_norm_grad(dy, x, w, g[0], workspace=ws), mf.layer_norm_grad(dy, x, w, g[1])) and torch.equal(g[0], g[1])
    with pytest.raises(mf.MfsdpError, match="WORKSPACE"):
        mf.layer_norm_grad(dy, x, w, g[0], workspace=ws[:1000])
    with pytest.raises(TypeError, match="must be a tensor"):
        mf.route_plan(e.to(DEV), 900, workspace=[1])


# ---------------------------------------------------------------------------
# Large
# ---------------------------------------------------------------------------
def test_rows_past_four_gib():
    # the last rows of buffers of more than 2^32 bytes are those of short ones
    d, tokens, k = 4096, 75000, 8
    rows = tokens * k                   # 4.9 GB of bf16
    place = torch.arange(rows, dtype=torch.int32, device=DEV).flip(0).view(tokens, k).contiguous()
    x, w = rand((1, d), BF, 1).to(DEV).repeat(tokens, 1), torch.rand(tokens, k, device=DEV)
    x[0], x[-1] = rand((d,), BF, 2).to(DEV), rand((d,), BF, 3).to(DEV)
    h = mf.route_dispatch(x, place)
    assert torch.equal(h[-k:], x[:1].expand(k, d)) and torch.equal(h[:k], x[-1:].expand(k, d)) and torch.equal(h[rows // 2], x[tokens // 2])
    y = mf.route_combine(h, place, w)
    short = mf.route_combine(h[-k:].contiguous(), place[:1] - (rows - k), w[:1])
    assert torch.equal(y[0], short[0])
    dh, dw = mf.route_combine_grad(x, h, place, w)
    sh, sw = mf.route_combine_grad(x[:1], h[-k:].contiguous(), place[:1] - (rows - k), w[:1])
    assert torch.equal(dh[-k:], sh) and torch.equal(dw[0], sw[0])
    del dh, y
    gain = torch.rand(d, device=DEV)
    n = mf.layer_norm(h, gain)
    assert torch.equal(n[-k:], mf.layer_norm(h[-k:].contiguous(), gain))
    del n
    dg = torch.empty(d, device=DEV)
    dx = mf.layer_norm_grad(h, h, gain, dg)
    assert torch.equal(dx[-k:], mf.layer_norm_grad(h[-k:].contiguous(), h[-k:].contiguous(), gain, torch.empty(d, device=DEV)))
    del dx
    both = torch.cat([h, h])            # 4.9 GB of codes
    codes, scales = mf.scaled_quantize(both)
    c, s = mf.scaled_quantize(both[-k:])
    assert torch.equal(codes[-k:].view(torch.uint8), c.view(torch.uint8)) and torch.equal(scales[-k:], s)
    wq = mf.scaled_quantize_weight(rand((1, 64, d), BF, 4, 0.05).to(DEV))
    y = mf.scaled_linear(codes, scales, *wq, torch.tensor([0, 2 * rows], dtype=torch.int32, device=DEV))
    one = mf.scaled_linear(c, s, *wq, torch.tensor([0, k], dtype=torch.int32, device=DEV))
    # other tiles add in another order: two roundings and the sums' own error
    assert float((y[-k:].double() - one.double()).norm() / one.double().norm()) <= 2 ** -8 + 2e-4


def test_many_tokens():
    # as many tokens as one launch may have, of one expert each
    t = (1 << 25) - 1
    x = torch.zeros(t, 2, device=DEV)
    x[::3, 1] = 1.0
    e, w = mf.route(x, 1)
    assert torch.equal(e[:, 0], (x[:, 1] > 0).to(torch.int32)) and float((w - 1).abs().max()) <= 2 ** -20
    p = mf.route_plan(e, 2)
    ones = (t + 2) // 3
    assert p.offsets.tolist() == [0, t - ones, t]
    assert torch.equal(p.place[::3, 0], torch.arange(t - ones, t, dtype=torch.int32, device=DEV))
    del x, w
    # one column: more tokens than one launch's workgroups take
    n = (1 << 24) * 4 + 5
    place = torch.arange(n, dtype=torch.int32, device=DEV).flip(0).view(n, 1).contiguous()
    v = torch.arange(n, device=DEV, dtype=torch.float32).view(n, 1)
    assert torch.equal(mf.route_dispatch(v, place), v.flip(0))
    assert torch.equal(mf.route_combine(v, place), v.flip(0))


def test_arguments():
    x, i = rand((4, 8), F32, 1).to(DEV), torch.zeros(4, 2, dtype=torch.int32, device=DEV)
    w = rand((8,), F32, 2).to(DEV)
    bad = [(ValueError, lambda: mf.route(x, 2, scores="tanh")), (ValueError, lambda: mf.route(x, 2, bias=w[:4])), (TypeError, lambda: mf.route(x, 2, bias=w.double())),
           (TypeError, lambda: mf.route(x, 2, mask=torch.ones(4, device=DEV))), (ValueError, lambda: mf.route(x.t(), 2)), (TypeError, lambda: mf.route(x.half(), 2)),
           (mf.MfsdpError, lambda: mf.route(x, 9)), (mf.MfsdpError, lambda: mf.route(x, 2, groups=3)), (ValueError, lambda: mf.route_grad(x, x, i)),
           (TypeError, lambda: mf.route_plan(i.long(), 3)), (ValueError, lambda: mf.route_dispatch(x, i[:3])), (ValueError, lambda: mf.route_combine(x, i, beta=1.0)),
           (ValueError, lambda: mf.route_combine(x, i, x)), (TypeError, lambda: mf.route_combine_grad(x.to(BF), x, i, x[:, :2].contiguous())),
           (ValueError, lambda: mf.layer_norm(x, w[:4])), (TypeError, lambda: mf.layer_norm(x, w, w.to(BF))), (mf.MfsdpError, lambda: mf.layer_norm(x, w, out=x)),
           (TypeError, lambda: mf.layer_norm_grad(x, x, w, w.to(BF))), (mf.MfsdpError, lambda: mf.layer_norm_grad(x, x, w, w)),
           (ValueError, lambda: mf.layer_norm(x.cpu(), w)), (ValueError, lambda: mf.layer_norm(x, w.cpu())), (TypeError, lambda: mf.scaled_quantize(x, codes=x)),
           (TypeError, lambda: mf.scaled_quantize_weight([1])), (ValueError, lambda: mf.scaled_quantize_weight(x))]
    q, qw = mf.scaled_quantize(x), mf.scaled_quantize_weight(x[None])
    off = torch.tensor([0, 4], dtype=torch.int32, device=DEV)
    bad += [(ValueError, lambda: mf.scaled_linear(q[0][:, :64], q[1], *qw, off)), (TypeError, lambda: mf.scaled_linear(q[0].view(torch.uint8), q[1], *qw, off)),
            (ValueError, lambda: mf.scaled_linear(*q, *qw, off[:1])), (TypeError, lambda: mf.scaled_linear(*q, *qw, off, out=torch.zeros(4, 4, device=DEV)))]
    for kind, f in bad:
        with pytest.raises(kind):
            f()


def test_timing_kinds():
    x, w = rand((8, 16), F32, 1).to(DEV), torch.ones(16, device=DEV)
    mf.timing.enable(True)
    try:
        mf.timing.reset()
        e, wt = mf.route(x, 2)
        p = mf.route_plan(e, 16)
        mf.route_combine(mf.route_dispatch(x, p.place), p.place, wt)
        mf.layer_norm_grad(x, x, w, torch.empty(16, device=DEV))
        mf.scaled_quantize(x)
        assert [mf.timing.read(kind)[1] for kind in ("route", "exchange", "layer_norm", "scaled")] == [2, 2, 2, 1]
    finally:
        mf.timing.enable(False)
        mf.timing.reset()
