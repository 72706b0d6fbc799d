"""What a rank runs on the flat buffers beside the step, in cases of real work: the embedding lookup and its gradient,
layer norm and RMS norm with their gradients, and activation checkpoints in 8 bits with their use in the backward pass.

Embedding (zf_embedding, zf_embedding_grad).  out[t] = scale table[ids[t]]; the gradient of row v is scale times the
sum of dout[t] over the tokens t with ids[t] = v, stored or added to what the row holds.  A token whose id lies outside
the vocabulary (-1 marks padding) takes a row of zeros and gives no gradient.

Norm (zf_layer_norm, zf_layer_norm_grad).  Per row, with r = 1 / sqrt(var + eps) and xh = (x - mean) r (RMS: mean = 0),
  y = xh w + b;   with h = dy w,  dx = r (h - avg(h) - xh avg(h xh)) (RMS: no avg(h)),  dw = sum dy xh,  db = sum dy.

Checkpoint (zf_act8_store, zf_act8_load).  Every 32 elements of a row share a power of two 2^k, k the least integer from
-100 on with amax <= 448 2^k over the finite ones, and are kept as e4m3 of x / 2^k, rounded to nearest, ties to even (a
value that would be rounded past its type's largest takes the largest code below).  zf_layer_norm writes checkpoints of
x and y in the same pass, zf_layer_norm_grad reads x from one, and zf_weight_grad is a Linear's dW = dY^T X from one.
"""
import math

import torch

own = False

DTYPES = {"f16": torch.float16, "bf16": torch.bfloat16, "f32": torch.float32}
SIZE = {"f16": 2, "bf16": 2, "f32": 4}
TOP = {torch.float16: 8, torch.bfloat16: 120, torch.float32: 120}  # the largest k that a type's values reach
EPS, GROUP = 1e-5, 32


# ---- the cases -----------------------------------------------------------------------------------------------------

def _embedding(name, n, vocab, cols, table, out, scale, wide):
    return {"name": name, "op": "embedding", "n": n, "vocab": vocab, "cols": cols, "table": table, "out": out,
            "scale": scale, "wide": wide}


def _embedding_grad(name, n, vocab, cols, dout, grad, scale, accumulate, wide):
    return {"name": name, "op": "embedding grad", "n": n, "vocab": vocab, "cols": cols, "dout": dout, "grad": grad,
            "scale": scale, "accumulate": accumulate, "wide": wide}


def _norm(name, kind, rows, cols, dtype, weight, bias, keep, gap):
    return {"name": name, "op": "norm", "kind": kind, "rows": rows, "cols": cols, "dtype": dtype, "weight": weight,
            "bias": bias, "keep": keep, "gap": gap}


def _norm_grad(name, kind, rows, cols, dtype, weight, bias, x, grad, accumulate, gap):
    return {"name": name, "op": "norm grad", "kind": kind, "rows": rows, "cols": cols, "dtype": dtype,
            "weight": weight, "bias": bias, "x": x, "grad": grad, "accumulate": accumulate, "gap": gap}


def _checkpoint(name, rows, cols, dtype, gap):
    return {"name": name, "op": "checkpoint", "rows": rows, "cols": cols, "dtype": dtype, "gap": gap}


def _weight_grad(name, rows, outs, ins, dtype, grad, accumulate, gap):
    return {"name": name, "op": "weight grad", "rows": rows, "out": outs, "in": ins, "dtype": dtype, "grad": grad,
            "accumulate": accumulate, "gap": gap}


def listed():
    return [
        # one short sequence through the table of the decoder of hidden size 1024: latency counts
        _embedding("lookup of 128 tokens", 128, 1024, 1024, "bf16", "bf16", 32.0, True),
        # 32768 tokens from the fp32 master shards of a per-parameter plan, hidden 2048, vocabulary 40960
        _embedding("lookup from fp32", 32768, 40960, 2048, "f32", "bf16", 1.0, False),
        # the gradient of a small table, stored into an fp32 buffer: every row is written
        _embedding_grad("table grad small", 1000, 1024, 1024, "bf16", "f32", 32.0, False, True),
        # a micro-batch of 32768 tokens added to the fp32 main gradients; frequent tokens fill whole tiles
        _embedding_grad("table grad added", 32768, 40960, 2048, "bf16", "f32", 1.0, True, False),
        # layer norm of a small batch of odd width between wider rows, both checkpoints: latency and ragged groups
        _norm("norm odd", "layer", 333, 1000, "f16", "f16", True, "xy", 3),
        # the decoder's RMS norm over 32768 tokens of hidden 2048, with its checkpoints
        _norm("norm h2048 kept", "rms", 32768, 2048, "bf16", "bf16", False, "xy", 0),
        # the backward pass of one sequence of 1000 tokens, hidden 1024, from full activations into the 16-bit replica
        _norm_grad("norm grad h1024", "layer", 1000, 1024, "bf16", "bf16", True, "full", "bf16", False, 0),
        # the same pass over 32768 tokens of hidden 2048 from a checkpoint, added to the fp32 main gradients
        _norm_grad("norm grad h2048 kept", "rms", 32768, 2048, "bf16", "bf16", False, "kept", "f32", True, 0),
        # an MLP's inner activations, 8192 wide, into 8 bits and back
        _checkpoint("checkpoint 8192", 8192, 8192, "bf16", 0),
        # a hidden layer of a small MLP of odd widths, strided gradients
        _weight_grad("dW odd", 333, 777, 1000, "f16", "f16", False, 3),
        # a key projection of the decoder of hidden 1024 over 16384 tokens: few tiles, long sums
        _weight_grad("dW 256x1024", 16384, 256, 1024, "bf16", "bf16", False, 0),
        # an up projection of hidden 2048 over 16384 tokens, added to the fp32 main gradients
        _weight_grad("dW 8192x2048", 16384, 8192, 2048, "bf16", "f32", True, 0),
    ]


def _spread(rng, lo, hi):
    """A whole number between lo and hi, even over its logarithm."""
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def _width(rng, hi):
    """Of layers: any number, or a multiple of 64."""
    w = _spread(rng, 1, hi)
    return max(64, w // 64 * 64) if rng.random() < 0.5 else w


def draw(rng):
    op = rng.choice(["embedding", "embedding grad", "norm", "norm grad", "checkpoint", "weight grad"])
    t, weight = rng.choice(["bf16", "bf16", "f16", "f32"]), rng.choice(["same", "f32"])
    weight, gap, accumulate = (t if weight == "same" else "f32"), rng.choice([0, 0, 1, 8]), rng.random() < 0.5
    if op in ("embedding", "embedding grad"):
        cols = _width(rng, 8192)
        vocab, n = _spread(rng, 1, min(131072, 40960 * 2048 // cols)), _spread(rng, 1, min(65536, 2 ** 25 // cols))
        scale, wide = rng.choice([1.0, round(math.sqrt(cols), 3)]), rng.random() < 0.5
        if op == "embedding":
            case = _embedding("", n, vocab, cols, rng.choice([t, "f32"]), t, scale, wide)
        else:
            case = _embedding_grad("", n, vocab, cols, t, rng.choice([t, "f32"]), scale, accumulate, wide)
    elif op == "weight grad":
        outs, ins = _width(rng, 8192), _width(rng, 8192)
        rows = _spread(rng, 1, min(32768, 2 ** 37 // (outs * ins)))
        t = rng.choice(["bf16", "f16"])
        case = _weight_grad("", rows, outs, ins, t, rng.choice([t, "f32"]), accumulate, gap)
    else:
        cols = _width(rng, 16384)
        rows = _spread(rng, 1, min(65536, 2 ** 25 // cols))
        kind, bias = rng.choice(["layer", "rms"]), rng.random() < 0.5
        if op == "norm":
            case = _norm("", kind, rows, cols, t, weight, bias, rng.choice(["", "x", "xy"]), gap)
        elif op == "norm grad":
            case = _norm_grad("", kind, rows, cols, t, weight, bias, rng.choice(["full", "kept"]),
                              rng.choice([t, "f32"]), accumulate, gap)
        else:
            case = _checkpoint("", rows, cols, t, gap)
    del case["name"]
    return case


# ---- inputs --------------------------------------------------------------------------------------------------------

def _chances(vocab):
    """Word frequencies: the k-th most frequent token in proportion to 1 / (k + 2)."""
    p = 1.0 / (torch.arange(vocab, dtype=torch.float64) + 3.0)
    return p / p.sum()


def _ids(g, case):
    """Tokens by word frequency over a shuffled vocabulary, 2% of them padding."""
    order = torch.randperm(case["vocab"], generator=g, device="cuda")
    ends = _chances(case["vocab"]).cumsum(0).cuda()
    at = torch.searchsorted(ends, torch.rand(case["n"], generator=g, device="cuda", dtype=torch.float64))
    ids = order[at.clamp(max=case["vocab"] - 1)]
    ids[torch.rand(case["n"], generator=g, device="cuda") < 0.02] = -1
    return ids if case["wide"] else ids.to(torch.int32)


def _rows(rows, cols, gap, dtype):
    """A matrix whose rows lie `gap` elements apart."""
    return torch.zeros(rows, cols + gap, dtype=dtype, device="cuda")[:, :cols]


def _activations(g, rows, cols, gap, dtype):
    """Unit deviation with an offset a row, and one channel in a hundred or so twenty times as large."""
    x = torch.randn(rows, cols, generator=g, device="cuda") + torch.randn(rows, 1, generator=g, device="cuda") * 0.3
    x *= torch.where(torch.rand(cols, generator=g, device="cuda") < 0.01, 20.0, 1.0)
    out = _rows(rows, cols, gap, dtype)
    return out.copy_(x)


def _upstream(g, rows, cols, gap, dtype):
    """Gradients of activations, loss-scaled in fp16."""
    out = _rows(rows, cols, gap, dtype)
    return out.copy_(torch.randn(rows, cols, generator=g, device="cuda") * (1.0 if dtype == torch.float16 else 1e-3))


def _held(g, shape, dtype, accumulate):
    """The gradient buffer: what earlier micro-batches left, or anything where it is written over."""
    return (torch.randn(shape, generator=g, device="cuda") * 1e-2).to(dtype) if accumulate else torch.full(
        shape, 7.0, dtype=dtype, device="cuda")


def _inputs(case, seed):
    g, op = torch.Generator(device="cuda").manual_seed(seed), case["op"]
    if op in ("embedding", "embedding grad"):
        made = {"ids": _ids(g, case)}
        if op == "embedding":
            table = torch.randn(case["vocab"], case["cols"], generator=g, device="cuda") * 0.02
            made["table"] = table.to(DTYPES[case["table"]])
        else:
            made["dout"] = _upstream(g, case["n"], case["cols"], 0, DTYPES[case["dout"]])
            made["grad"] = _held(g, (case["vocab"], case["cols"]), DTYPES[case["grad"]], case["accumulate"])
        return made
    if op == "weight grad":
        made = {"dy": _upstream(g, case["rows"], case["out"], case["gap"], DTYPES[case["dtype"]]),
                "x": _activations(g, case["rows"], case["in"], 0, DTYPES[case["dtype"]])}
        made["grad"] = _held(g, (case["out"], case["in"]), DTYPES[case["grad"]], case["accumulate"])
        return made
    dt, rows, cols = DTYPES[case["dtype"]], case["rows"], case["cols"]
    made = {"x": _activations(g, rows, cols, case["gap"], dt)}
    if op == "checkpoint":
        return made
    made["weight"] = (1.0 + 0.1 * torch.randn(cols, generator=g, device="cuda")).to(DTYPES[case["weight"]])
    made["bias"] = (0.1 * torch.randn(cols, generator=g, device="cuda")).to(DTYPES[case["weight"]]) if case[
        "bias"] else None
    if op == "norm grad":
        made["dy"] = _upstream(g, rows, cols, case["gap"], dt)
        mean, rstd = _statistics(made["x"].double(), case["kind"])
        made["mean"], made["rstd"] = mean.float().reshape(-1) if case["kind"] == "layer" else None, rstd.float().reshape(-1)
        gt = DTYPES[case["grad"]]
        made["weight_grad"] = _held(g, (cols,), gt, case["accumulate"])
        made["bias_grad"] = _held(g, (cols,), gt, case["accumulate"]) if case["bias"] else None
    return made


def _blank8(rows, cols):
    """The buffers of a checkpoint: codes and a scale for each 32 elements of a row."""
    return (torch.zeros(rows, cols, dtype=torch.uint8, device="cuda"),
            torch.zeros(rows, -(-cols // GROUP), dtype=torch.uint8, device="cuda"))


def prepare(case, seed):
    made, op = _inputs(case, seed), case["op"]
    made["case"] = case
    if op == "embedding":
        made["out"] = torch.empty(case["n"], case["cols"], dtype=DTYPES[case["out"]], device="cuda")
    elif op == "norm":
        rows, cols = made["x"].shape
        made["y"] = _rows(rows, cols, case["gap"], made["x"].dtype)
        made["mean"] = torch.empty(rows, device="cuda") if case["kind"] == "layer" else None
        made["rstd"] = torch.empty(rows, device="cuda")
        made["x8"] = _blank8(rows, cols) if "x" in case["keep"] else None
        made["y8"] = _blank8(rows, cols) if "y" in case["keep"] else None
    elif op == "norm grad":
        made["dx"] = _rows(*made["x"].shape, case["gap"], made["x"].dtype)
        if case["x"] == "kept":
            made["x8"] = _store(made.pop("x"))
    elif op == "checkpoint":
        made["x8"] = _blank8(*made["x"].shape)
        made["back"] = torch.empty(made["x"].shape, dtype=made["x"].dtype, device="cuda")
    elif op == "weight grad":
        made["x8"] = _store(made.pop("x"))
    if own:  # the workspace and the checkpoints' handles that a program keeps
        from fsdp_sharded_mixed_amd import zf
        need = 0
        if op == "embedding grad":
            need = zf.embedding_grad_bytes(case["n"], case["vocab"], case["cols"])
        elif op == "norm grad":
            need = zf.layer_norm_grad_bytes(case["rows"], case["cols"])
        elif op == "weight grad":
            need = zf.weight_grad_bytes(case["rows"], case["out"], case["in"])
        made["workspace"] = torch.empty(need, dtype=torch.uint8, device="cuda")
        for key in ("x8", "y8"):
            made["h" + key] = zf.act8(*made[key]) if made.get(key) else None
    return made


# ---- the plain forms -----------------------------------------------------------------------------------------------

def _groups(x, fill):
    """[rows, groups, 32], the last group of a row filled up."""
    return torch.nn.functional.pad(x, (0, -x.shape[1] % GROUP), value=fill).view(x.shape[0], -1, GROUP)


def _power(k):
    """2^k in 32 bits, by its bits, for whole k from -126 to 127: exact, which pow() is not."""
    return ((k.int() + 127) << 23).view(torch.float32)


def _store(x):
    """The checkpoint of x: (codes, scales) as bytes."""
    v = _groups(x.float(), 0.0)
    fine = torch.isfinite(v)
    top = torch.where(fine, v.abs(), 0.0).amax(2)
    part, power = torch.frexp(top)  # top = part 2^power, part in [1/2, 1)
    k = torch.where(part <= 0.875, power - 9, power - 8).clamp(min=-100)
    k = torch.where(top == 0, -100, k)
    most = torch.where(k == TOP[x.dtype], 240.0, 448.0)[:, :, None]
    small = (torch.where(fine, v, 0.0) * _power(-k)[:, :, None]).clamp(-most, most)
    codes = torch.where(fine, small, math.nan).to(torch.float8_e4m3fn).view(torch.uint8)
    codes = torch.where(fine, codes, 0x7F)
    return codes.view(x.shape[0], -1)[:, :x.shape[1]].contiguous(), (k + 127).to(torch.uint8)


def _load(kept):
    """What a checkpoint stands for, in 32 bits."""
    codes, scales = kept
    v = _groups(codes, 0).view(torch.float8_e4m3fn).float() * _power(scales.int() - 127)[:, :, None]
    return v.view(codes.shape[0], -1)[:, :codes.shape[1]]


def _statistics(x, kind):
    mean = x.mean(1, keepdim=True) if kind == "layer" else torch.zeros(x.shape[0], 1, dtype=x.dtype, device=x.device)
    return mean, 1.0 / torch.sqrt((x - mean).square().mean(1, keepdim=True) + EPS)


def _write(grad, new, accumulate):
    return grad.copy_(grad.float() + new if accumulate else new)


def _plain(s):
    case = s["case"]
    op = case["op"]
    if op == "embedding":
        rows = s["table"][s["ids"].long().clamp(min=0)].float() * case["scale"]
        s["out"].copy_(torch.where((s["ids"] >= 0)[:, None], rows, 0.0))
    elif op == "embedding grad":
        at = torch.where(s["ids"] >= 0, s["ids"].long(), case["vocab"])
        total = torch.zeros(case["vocab"] + 1, case["cols"], device="cuda").index_add_(0, at, s["dout"].float())
        _write(s["grad"], total[:-1] * case["scale"], case["accumulate"])
    elif op == "norm":
        x = s["x"].float()
        mean, rstd = _statistics(x, case["kind"])
        y = (x - mean) * rstd * s["weight"].float()
        s["y"].copy_(y + s["bias"].float() if case["bias"] else y)
        s["rstd"].copy_(rstd.view(-1))
        if s["mean"] is not None:
            s["mean"].copy_(mean.view(-1))
        for kept, v in ((s["x8"], s["x"]), (s["y8"], s["y"])):
            if kept is not None:
                codes, scales = _store(v)
                kept[0].copy_(codes)
                kept[1].copy_(scales)
    elif op == "norm grad":
        x = _load(s["x8"]) if case["x"] == "kept" else s["x"].float()
        dy, r = s["dy"].float(), s["rstd"][:, None]
        xh = (x - s["mean"][:, None] if s["mean"] is not None else x) * r
        h = dy * s["weight"].float()
        dx = h - xh * (h * xh).mean(1, keepdim=True)
        s["dx"].copy_(r * (dx - h.mean(1, keepdim=True) if case["kind"] == "layer" else dx))
        _write(s["weight_grad"], (dy * xh).sum(0), case["accumulate"])
        if case["bias"]:
            _write(s["bias_grad"], dy.sum(0), case["accumulate"])
    elif op == "checkpoint":
        codes, scales = _store(s["x"])
        s["x8"][0].copy_(codes)
        s["x8"][1].copy_(scales)
        s["back"].copy_(_load(s["x8"]))
    else:
        _write(s["grad"], s["dy"].float().t() @ _load(s["x8"]), case["accumulate"])


def _kept(pair):
    """A checkpoint's two parts as the numbers that they stand for: e4m3, and powers of two."""
    return None if pair is None else (pair[0].view(torch.float8_e4m3fn), pair[1].view(torch.float8_e8m0fnu))


def _answer(s):
    op = s["case"]["op"]
    if op == "embedding":
        return {"out": s["out"]}
    if op == "norm":
        return {"y": s["y"], "mean": s["mean"], "rstd": s["rstd"], "x8": _kept(s["x8"]), "y8": _kept(s["y8"])}
    if op == "norm grad":
        return {"dx": s["dx"], "weight_grad": s["weight_grad"], "bias_grad": s["bias_grad"]}
    if op == "checkpoint":
        return {"x8": _kept(s["x8"]), "back": s["back"]}
    return {"grad": s["grad"]}


def run(s):
    if not own:
        _plain(s)
        return _answer(s)
    from fsdp_sharded_mixed_amd import zf
    case = s["case"]
    op = case["op"]
    if op == "embedding":
        zf.embedding(s["table"], s["ids"], s["out"], scale=case["scale"])
    elif op == "embedding grad":
        zf.embedding_grad(s["dout"], s["ids"], s["grad"], s["workspace"], scale=case["scale"],
                          accumulate=case["accumulate"])
    elif op == "norm":
        kind = zf.NORM_LAYER if case["kind"] == "layer" else zf.NORM_RMS
        zf.layer_norm(kind, s["x"], s["weight"], s["bias"], EPS, s["y"], s["mean"], s["rstd"], x8=s["hx8"],
                      y8=s["hy8"])
    elif op == "norm grad":
        kind = zf.NORM_LAYER if case["kind"] == "layer" else zf.NORM_RMS
        zf.layer_norm_grad(kind, s["dy"], s["hx8"] if case["x"] == "kept" else s["x"], s["weight"], s["mean"],
                           s["rstd"], s["dx"], s["weight_grad"], s["bias_grad"], s["workspace"],
                           accumulate=case["accumulate"])
    elif op == "checkpoint":
        zf.act8_store(s["hx8"], s["x"])
        zf.act8_load(s["hx8"], s["back"])
    else:
        zf.weight_grad(s["dy"], s["hx8"], s["grad"], s["workspace"], accumulate=case["accumulate"])
    return _answer(s)


# ---- the work ------------------------------------------------------------------------------------------------------

def _distinct(case):
    """The rows of the table that a batch is expected to touch."""
    return float((1.0 - (1.0 - 0.98 * _chances(case["vocab"])) ** case["n"]).sum())


def work(case):
    op = case["op"]
    if op in ("embedding", "embedding grad"):
        n, cols, ids = case["n"], case["cols"], case["n"] * (8 if case["wide"] else 4)
        if op == "embedding":
            return {"bytes": ids + cols * (n * SIZE[case["out"]] + _distinct(case) * SIZE[case["table"]]),
                    "flops": n * cols}
        rows = 2 * _distinct(case) if case["accumulate"] else case["vocab"]
        return {"bytes": ids + cols * (n * SIZE[case["dout"]] + rows * SIZE[case["grad"]]), "flops": n * cols}
    if op == "weight grad":
        size = case["out"] * case["in"]
        kept = case["in"] + -(-case["in"] // GROUP)
        return {"bytes": case["rows"] * (case["out"] * SIZE[case["dtype"]] + kept)
                + size * SIZE[case["grad"]] * (2 if case["accumulate"] else 1), "flops": 2 * case["rows"] * size}
    rows, cols, size = case["rows"], case["cols"], SIZE[case["dtype"]]
    kept, total = rows * (cols + -(-cols // GROUP)), rows * cols
    if op == "checkpoint":  # written, then read again
        return {"bytes": 2 * total * size + 2 * kept, "flops": 4 * total}
    stats, vectors = rows * (8 if case["kind"] == "layer" else 4), cols * (2 if case["bias"] else 1)
    if op == "norm":
        return {"bytes": 2 * total * size + kept * len(case["keep"]) + stats + vectors * SIZE[case["weight"]],
                "flops": 7 * total}
    return {"bytes": total * size * 2 + (kept if case["x"] == "kept" else total * size) + stats
            + cols * SIZE[case["weight"]] + vectors * SIZE[case["grad"]] * (2 if case["accumulate"] else 1),
            "flops": 12 * total}


# ---- the definition in 64 bits -------------------------------------------------------------------------------------

def _power_64(k):
    return ((k.long() + 1023) << 52).view(torch.float64)


def _scale_64(x):
    """k of every element of x, by trying: the least k >= -100 with the group's largest magnitude <= 448 2^k."""
    top = torch.where(torch.isfinite(x), x, 0.0).abs().double()
    pad = -x.shape[1] % GROUP
    top = torch.cat([top, top.new_zeros(x.shape[0], pad)], 1).view(x.shape[0], -1, GROUP).max(2).values
    k = torch.ceil(torch.log2(top.clamp(min=2.0 ** -140) / 448.0)) + 1
    for _ in range(3):
        k = torch.where((k > -100) & (top <= 448.0 * _power_64(k - 1)), k - 1, k)
    return k.clamp(min=-100)


def _code_64(x):
    """(e4m3 numbers, powers of two) of the checkpoint of x, whose values are finite."""
    k = _scale_64(x)
    every = k.repeat_interleave(GROUP, 1)[:, :x.shape[1]]
    v = x.double() / _power_64(every)
    step = _power_64(torch.frexp(v)[1].clamp(min=-5) - 4)  # three bits behind the first, none below 2^-9
    v = torch.round(v / step) * step
    return torch.where((every == TOP[x.dtype]) & (v.abs() > 240), 240.0 * v.sign(), v), _power_64(k)


def _kept_64(x):
    codes, powers = _code_64(x)
    return codes * powers.repeat_interleave(GROUP, 1)[:, :x.shape[1]]


def exact(case, seed):
    made, op = _inputs(case, seed), case["op"]
    if op == "embedding":
        out = torch.zeros(case["n"], case["cols"], dtype=torch.float64, device="cuda")
        real = made["ids"] >= 0
        out[real] = made["table"].double()[made["ids"][real].long()] * case["scale"]
        return {"out": out}
    if op == "embedding grad":
        real = made["ids"] >= 0
        ids, order = torch.sort(made["ids"][real].long(), stable=True)
        run = made["dout"][real][order].double().cumsum(0)  # sums of runs as differences of a running sum
        last = torch.ones_like(ids, dtype=torch.bool)
        last[:-1] = ids[1:] != ids[:-1]
        ends = run[last]
        grad = made["grad"].double() if case["accumulate"] else torch.zeros(
            case["vocab"], case["cols"], dtype=torch.float64, device="cuda")
        if len(ids):
            ends[1:] -= ends[:-1].clone()
            grad[ids[last]] += ends * case["scale"]
        return {"grad": grad}
    if op == "weight grad":
        grad = torch.mm(made["dy"].double().t(), _kept_64(made["x"]))
        return {"grad": grad + made["grad"].double() if case["accumulate"] else grad}
    if op == "checkpoint":
        return {"x8": _code_64(made["x"]), "back": _kept_64(made["x"])}
    x, w = made["x"].double(), made["weight"].double()
    if op == "norm":
        mean = x.sum(1) / x.shape[1] if case["kind"] == "layer" else None
        centred = x if mean is None else x - mean[:, None]
        rstd = (centred.pow(2).sum(1) / x.shape[1] + EPS) ** -0.5
        y = centred * rstd[:, None] * w
        # the checkpoint of y is that of y as its type holds it: a rounding away from this y has no value here
        return {"y": y if made["bias"] is None else y + made["bias"].double(), "mean": mean, "rstd": rstd,
                "x8": _code_64(made["x"]) if "x" in case["keep"] else None, "y8": None}
    x = _kept_64(made["x"]) if case["x"] == "kept" else x
    dy, rstd = made["dy"].double(), made["rstd"].double()
    if made["mean"] is not None:
        x = x - made["mean"].double()[:, None]
    cols, h = x.shape[1], dy * w
    along = (h * x).sum(1) * rstd ** 3 / cols  # avg(h xh) r^2, for x in place of xh
    dx = h * rstd[:, None] - x * along[:, None]
    if case["kind"] == "layer":
        dx = dx - (h.sum(1) * rstd / cols)[:, None]
    dw, db = torch.mv((dy * x).t(), rstd), dy.sum(0)
    if case["accumulate"]:
        dw = dw + made["weight_grad"].double()
        db = db + made["bias_grad"].double() if case["bias"] else None
    return {"dx": dx, "weight_grad": dw, "bias_grad": db if case["bias"] else None}
