"""Cases for the operators that make the gradients of the owner-local step.

* ``linear``: products grouped by expert, ``Y[r] = X[r] W_e^T`` for the rows
  ``offsets[e] <= r < offsets[e + 1]`` (forward).
* ``linear_grads``: their gradients, ``dX[r] = dY[r] W_e`` and
  ``dW_e = sum_r dY[r]^T X[r]``, the gradients that the Muon step takes.
* ``linear_grads_ckpt``: the same two with X kept as an 8-bit checkpoint.
* ``checkpoint``: an activation to its 8-bit checkpoint and back.
* ``embedding``: scaled table rows of a list of tokens.
* ``embedding_grad``: the table's dense fp32 gradient, which the AdamW tail takes.

An 8-bit checkpoint holds, for each row and each block of 128 columns, whole
numbers q in [-127, 127] and one power of two 2^e, the smallest with
max |x| <= 127 * 2^e: x is held as q * 2^e, q = x / 2^e rounded to the nearest,
ties to even (e is stored as e + 127 in a byte).  Tokens outside the table stand
for padding: their row is zero and they add no gradient.
"""

import math

import numpy as np
import torch

own = False

BLOCK = 128
DTYPES = {"bf16": torch.bfloat16, "fp32": torch.float32}
SIZE = {"bf16": 2, "fp32": 4}


def listed():
    return [
        # four tokens, two experts each, one decoding step of a small-expert layer (512 x 1536 experts)
        {"name": "linear decode", "kind": "linear", "dtype": "bf16", "experts": 256, "rows": 8, "n": 512, "k": 1536, "skew": 0.5},
        # a training batch over 256 small experts: ragged segments of about 128 rows
        {"name": "linear many small", "kind": "linear", "dtype": "bf16", "experts": 256, "rows": 32771, "n": 512, "k": 1536, "skew": 0.5},
        # a training batch over eight large experts (14336 x 4096)
        {"name": "grads large", "kind": "linear_grads", "dtype": "bf16", "experts": 8, "rows": 16384, "n": 14336, "k": 4096, "skew": 0.3},
        # an fp32 model of odd sizes: rows that start off every 16-byte boundary
        {"name": "grads odd fp32", "kind": "linear_grads", "dtype": "fp32", "experts": 7, "rows": 2049, "n": 513, "k": 257, "skew": 1.0},
        # 256 small experts whose inputs were kept in 8 bits
        {"name": "ckpt grads many small", "kind": "linear_grads_ckpt", "dtype": "bf16", "experts": 256, "rows": 32771, "n": 512, "k": 1536, "skew": 0.5},
        # sixteen experts of a d=2048 block, inputs kept in 8 bits
        {"name": "ckpt grads d2048", "kind": "linear_grads_ckpt", "dtype": "bf16", "experts": 16, "rows": 24576, "n": 5632, "k": 2048, "skew": 0.7},
        # the input of one d=5120 block's down projection
        {"name": "checkpoint d5120", "kind": "checkpoint", "dtype": "bf16", "rows": 8192, "k": 27648},
        # a short fp32 batch with a last block of 44 columns
        {"name": "checkpoint short", "kind": "checkpoint", "dtype": "fp32", "rows": 1000, "k": 300},
        # one decoding step of 32 sequences from an fp32 table
        {"name": "embedding decode", "kind": "embedding", "dtype": "bf16", "table": "fp32", "vocab": 32000, "d": 2048, "tokens": 32, "pad": 0.0},
        # a training batch, an eighth of it padding
        {"name": "embedding batch", "kind": "embedding", "dtype": "bf16", "table": "bf16", "vocab": 100000, "d": 4096, "tokens": 32768, "pad": 0.125},
        # its gradient, frequent tokens among the list some thousand times
        {"name": "embedding grad batch", "kind": "embedding_grad", "dtype": "bf16", "vocab": 100000, "d": 4096, "tokens": 32768, "pad": 0.125},
        # a short fp32 batch on a small table of an odd width
        {"name": "embedding grad short", "kind": "embedding_grad", "dtype": "fp32", "vocab": 5000, "d": 300, "tokens": 1000, "pad": 0.0},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _width(rng, lo, hi):
    """Mostly whole 16-byte rows, as models have them, and any number now and then."""
    v = _log(rng, lo, hi)
    return v if rng.random() < 0.25 else max(64, v // 64 * 64) if rng.random() < 0.7 else max(8, v // 8 * 8)


def draw(rng):
    kind = rng.choice(["linear", "linear", "linear_grads", "linear_grads", "linear_grads_ckpt", "checkpoint", "embedding", "embedding_grad"])
    dtype = rng.choice(["bf16", "bf16", "fp32"])
    if kind.startswith("linear"):
        while True:
            c = {"kind": kind, "dtype": dtype, "experts": _log(rng, 1, 256), "rows": _log(rng, 1, 32768),
                 "n": _width(rng, 64, 14336), "k": _width(rng, 64, 5632), "skew": round(rng.uniform(0.0, 1.0), 2)}
            if c["experts"] * c["n"] * c["k"] <= 4 * 10 ** 8 and c["rows"] * c["n"] * c["k"] <= (9 if dtype == "bf16" else 1) * 10 ** 11:
                return c
    if kind == "checkpoint":
        return {"kind": kind, "dtype": dtype, "rows": _log(rng, 1, 32768), "k": _width(rng, 64, 6912)}
    c = {"kind": kind, "dtype": dtype, "vocab": _log(rng, 1000, 100000), "d": _width(rng, 64, 4096), "tokens": _log(rng, 1, 32768),
         "pad": rng.choice([0.0, 0.1])}
    return dict(c, table=rng.choice(["bf16", "fp32"])) if kind == "embedding" else c


def _power(biased):
    """2^(biased - 127) exactly, from its bits (torch.ldexp multiplies by a pow that may be a bit off)."""
    return (biased.to(torch.int32) << 23).view(torch.float32)


def _quantize(x):
    """Plain 8-bit checkpoint of x: (codes int8, biased exponents uint8)."""
    rows, k = x.shape
    blocks = -(-k // BLOCK)
    v = torch.zeros(rows, blocks * BLOCK, dtype=torch.float32, device=x.device)
    v[:, :k] = x.float()
    v = v.view(rows, blocks, BLOCK)
    m, p = torch.frexp(v.abs().amax(2))                    # max = m * 2^p, m in [1/2, 1) or 0
    e = (p - 7 + (m > 127.0 / 128.0).to(p.dtype)).clamp(min=-126)
    e = torch.where(m == 0, torch.full_like(e, -126), e)
    q = torch.round(v * _power(127 - e)[:, :, None]).view(rows, blocks * BLOCK)[:, :k]
    return q.to(torch.int8).contiguous(), (e + 127).to(torch.uint8)


def _restore(codes, scales):
    return codes.float() * _power(scales).repeat_interleave(BLOCK, 1)[:, : codes.shape[1]]


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(int(seed))
    host = np.random.RandomState(int(seed) % (1 << 31))
    kind, dt = case["kind"], DTYPES[case["dtype"]]

    def normal(*shape):
        return torch.randn(*shape, generator=g, device="cuda")

    s = {"kind": kind, "dtype": dt}
    if kind.startswith("linear"):
        experts, rows, n, k = case["experts"], case["rows"], case["n"], case["k"]
        # routing: log-normal popularity of the experts, rows sorted by expert
        p = np.exp(case["skew"] * host.standard_normal(experts))
        counts = host.multinomial(rows, p / p.sum())
        s["counts"] = counts.tolist()
        s["longest"] = int(counts.max())
        s["offsets"] = torch.from_numpy(np.concatenate([[0], np.cumsum(counts)]).astype(np.int32)).cuda()
        s["w"] = torch.empty(experts, n, k, dtype=dt, device="cuda").normal_(0.0, 0.02, generator=g)
        s["x"] = x = normal(rows, k).to(dt)
        if kind != "linear":
            s["dy"] = (1e-3 * normal(rows, n)).to(dt)
            s["dw"] = torch.empty_like(s["w"])
        if kind == "linear_grads_ckpt":
            s["codes"], s["scales"] = _quantize(x)
            del s["x"]
    elif kind == "checkpoint":
        # activations: rows of different size, some columns far larger than the rest
        x = normal(case["rows"], case["k"]) * torch.exp(normal(case["rows"], 1))
        s["x"] = (x * torch.where(torch.rand(case["k"], generator=g, device="cuda") < 0.01, 30.0, 1.0)).to(dt)
    else:
        vocab, d, tokens = case["vocab"], case["d"], case["tokens"]
        # token frequency falls like 1 / rank; the ranks are spread over the table
        u = torch.rand(tokens, generator=g, device="cuda", dtype=torch.float64)
        rank = torch.exp(u * math.log(vocab)).to(torch.int64).clamp(max=vocab) - 1
        t = torch.randperm(vocab, generator=g, device="cuda")[rank]
        t = torch.where(torch.rand(tokens, generator=g, device="cuda") < case["pad"], -1, t)
        s["tokens"], s["vocab"], s["scale"] = t, vocab, math.sqrt(d)
        if kind == "embedding":
            s["table"] = (0.02 * normal(vocab, d)).to(DTYPES[case["table"]])
        else:
            s["dy"] = (1e-3 * normal(tokens, d)).to(dt)
            s["grad"] = torch.empty(vocab, d, device="cuda")
    return s


def _places(s):
    """Padded layout of the ragged rows: row of (expert, place), which places hold one, and each row's expert and place."""
    off = s["offsets"].to(torch.int64)
    place = torch.arange(s["longest"], device=off.device)
    row = off[:-1, None] + place
    held = row < off[1:, None]
    row = torch.where(held, row, 0)
    r = torch.arange(s["dy" if "dy" in s else "x"].shape[0], device=off.device)
    expert = torch.searchsorted(off[1:].contiguous(), r, right=True)
    return row, held, expert, r - off[expert]


def _plain_linear(s):
    row, held, expert, place = _places(s)
    x = torch.where(held[:, :, None], s["x"][row].float(), 0.0)
    return torch.bmm(x, s["w"].float().transpose(1, 2))[expert, place].to(s["dtype"])


def _plain_linear_grads(s):
    row, held, expert, place = _places(s)
    x = s["x"].float() if "x" in s else _restore(s["codes"], s["scales"])
    dy = torch.where(held[:, :, None], s["dy"][row].float(), 0.0)
    dx = torch.bmm(dy, s["w"].float())[expert, place].to(s["dtype"])
    dw = torch.bmm(dy.transpose(1, 2), torch.where(held[:, :, None], x[row], 0.0)).to(s["dtype"])
    return {"dx": dx, "dw": dw}


def _plain_embedding(s):
    t, held = s["tokens"], (s["tokens"] >= 0) & (s["tokens"] < s["vocab"])
    rows = s["table"][torch.where(held, t, 0)].float() * s["scale"]
    return torch.where(held[:, None], rows, 0.0).to(s["dtype"])


def _plain_embedding_grad(s):
    t, held = s["tokens"], (s["tokens"] >= 0) & (s["tokens"] < s["vocab"])
    rows = torch.where(held[:, None], s["dy"].float(), 0.0)
    return torch.zeros_like(s["grad"]).index_add_(0, torch.where(held, t, 0), rows) * s["scale"]


def run(state):
    s = state
    kind = s["kind"]
    if own:
        import matrix_optimizer_step_owner_amd as mf
        if kind == "linear":
            return mf.grouped_linear(s["x"], s["w"], s["offsets"])
        if kind == "linear_grads":
            dx = mf.grouped_linear_dgrad(s["dy"], s["w"], s["offsets"])
            return {"dx": dx, "dw": mf.grouped_linear_wgrad(s["dy"], s["x"], s["offsets"], s["dw"])}
        if kind == "linear_grads_ckpt":
            dx = mf.grouped_linear_dgrad(s["dy"], s["w"], s["offsets"])
            return {"dx": dx, "dw": mf.grouped_linear_wgrad_ckpt(s["dy"], s["codes"], s["scales"], s["offsets"], s["dw"])}
        if kind == "checkpoint":
            codes, scales = mf.ckpt_quantize(s["x"])
            return mf.ckpt_restore(codes, scales, s["dtype"])
        if kind == "embedding":
            return mf.embedding(s["table"], s["tokens"], scale=s["scale"], dtype=s["dtype"])
        return mf.embedding_grad(s["dy"], s["tokens"], s["grad"], scale=s["scale"])
    if kind == "linear":
        return _plain_linear(s)
    if kind.startswith("linear_grads"):
        return _plain_linear_grads(s)
    if kind == "checkpoint":
        return _restore(*_quantize(s["x"])).to(s["dtype"])
    return _plain_embedding(s) if kind == "embedding" else _plain_embedding_grad(s)


def work(case):
    kind, z = case["kind"], SIZE[case["dtype"]]
    if kind.startswith("linear"):
        m, n, k, e = case["rows"], case["n"], case["k"], case["experts"]
        if kind == "linear":    # experts without rows need not be read
            return {"bytes": z * (m * k + m * n + min(e, m) * n * k), "flops": 2 * m * n * k}
        held = m * k * z if kind == "linear_grads" else m * (k + -(-k // BLOCK))
        return {"bytes": z * (m * n + m * k + (min(e, m) + e) * n * k) + held, "flops": 4 * m * n * k}
    if kind == "checkpoint":    # read, kept, read again, written
        m, k = case["rows"], case["k"]
        return {"bytes": 2 * m * k * z + 2 * m * (k + -(-k // BLOCK)), "flops": 3 * m * k}
    t, d, v = case["tokens"], case["d"], case["vocab"]
    if kind == "embedding":
        return {"bytes": min(t, v) * d * SIZE[case["table"]] + t * (d * z + 8), "flops": t * d}
    return {"bytes": t * (d * z + 8) + v * d * 4, "flops": 2 * t * d}


def _power64(e):
    return ((e.to(torch.int64) + 1023) << 52).view(torch.float64)


def exact(case, seed):
    s = prepare(case, seed)
    kind = s["kind"]
    if kind.startswith("linear"):
        if "x" in s:
            x = s["x"].double()
        else:
            x = s["codes"].double()
            for b in range(s["scales"].shape[1]):
                x[:, b * BLOCK:(b + 1) * BLOCK] *= _power64(s["scales"][:, b:b + 1].to(torch.int64) - 127)
        y, dx, dw, at = [], [], [], 0
        for e, m in enumerate(s["counts"]):
            w = s["w"][e].double()
            if kind == "linear":
                y.append(x[at:at + m] @ w.t())
            else:
                d = s["dy"][at:at + m].double()
                dx.append(d @ w)
                dw.append(d.t() @ x[at:at + m])
            at += m
        return torch.cat(y) if kind == "linear" else {"dx": torch.cat(dx), "dw": torch.stack(dw)}
    if kind == "checkpoint":
        x = s["x"].double()
        for b in range(0, x.shape[1], BLOCK):
            v = x[:, b:b + BLOCK]
            top = v.abs().amax(1, keepdim=True).clamp(min=127.0 * 2.0 ** -126)
            e = torch.floor(torch.log2(top)) - 8    # at or below the smallest: at most three steps up
            e = torch.where(top > 127.0 * _power64(e), e + 1, e)
            e = torch.where(top > 127.0 * _power64(e), e + 1, e)
            e = _power64(torch.where(top > 127.0 * _power64(e), e + 1, e))
            x[:, b:b + BLOCK] = torch.round(v / e) * e
        return x
    t = s["tokens"]
    held = ((t >= 0) & (t < s["vocab"])).nonzero()[:, 0]
    if kind == "embedding":
        out = torch.zeros(t.numel(), s["table"].shape[1], dtype=torch.float64, device=t.device)
        out[held] = s["table"][t[held]].double() * s["scale"]
        return out
    return torch.zeros(s["grad"].shape, dtype=torch.float64, device=t.device).index_add_(0, t[held], s["dy"][held].double() * s["scale"])
