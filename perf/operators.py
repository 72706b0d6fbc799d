"""The Muon operators in cases of real work: orthogonalising a batch of update matrices, and the sharded Muon step.

Orthogonalisation (zf_orthogonalize).  For every matrix G of a batch, with m = min(rows, cols) and n = max(rows, cols),
  X = G / (|G|_F + eps), transposed where rows > cols, then `steps` times
  A = X X^T,  X <- a X + (b A + c A A) X,
and X (transposed back) is the result: the singular values of G are driven towards one, the singular vectors kept.

The sharded Muon step (zf_muon_step).  N replicas' 16-bit gradients in the padded flat layout are summed in rank order
in 32 bits, a non-finite sum skips the step, gs = coef / (S N) removes the loss scale, averages and clips by the global
norm; then, for every matrix that the plan gives to Muon,
  M <- mu M + g,  U = g + mu M (Nesterov) or M,  O = orthogonalised U,  W <- W (1 - lr wd) - lr scale O,
scale = sqrt(max(1, rows / cols)) or 0.2 sqrt(max(rows, cols)), and AdamW for every other parameter; the 16-bit
parameters are the rounded masters.
"""
import math

import torch

own = False

NS = (3.4445, -4.7750, 2.0315)  # a, b, c of the quintic step
NS_STEPS, NS_EPS = 5, 1e-7
DTYPES = {"f16": torch.float16, "bf16": torch.bfloat16, "f32": torch.float32}
LAYOUTS = {"global flat": 0, "per unit": 1, "per parameter": 2}
BETA1, BETA2, EPS, DECAY, MOMENTUM, MAX_NORM = 0.9, 0.999, 1e-8, 0.01, 0.95, 1.0


# ---- the cases ---------------------------------------------------------------------------------------------------

def _ortho(name, shapes, src, dst, gap=0):
    return {"name": name, "op": "orthogonalize", "shapes": shapes, "src": src, "dst": dst, "gap": gap}


def _decoder(name, hidden, inter, q, kv, layers, vocab, ranks, layout, grad, param, lr, scale, nesterov, reduced):
    return {"name": name, "op": "muon", "model": "decoder", "hidden": hidden, "inter": inter, "q": q, "kv": kv,
            "layers": layers, "vocab": vocab, "ranks": ranks, "layout": layout, "grad": grad, "param": param, "lr": lr,
            "scale": scale, "nesterov": nesterov, "reduced": reduced}


def _mlp(name, widths, ranks, layout, grad, param, lr, scale, nesterov, reduced):
    return {"name": name, "op": "muon", "model": "mlp", "widths": widths, "ranks": ranks, "layout": layout,
            "grad": grad, "param": param, "lr": lr, "scale": scale, "nesterov": nesterov, "reduced": reduced}


def listed():
    return [
        # the five weights of a small MLP: the call's latency counts
        _ortho("mlp weights", "128x40,128x128,64x128,32x64,16x34", "f32", "bf16"),
        # one projection of a decoder of hidden size 1024, alone on the GPU
        _ortho("one projection", "1024x1024", "bf16", "bf16"),
        # uneven matrices cut out of wider buffers: a row, a column, odd sizes, both orientations
        _ortho("odd shapes", "1x77,65x1,257x1000,1000x333,130x4097,999x1001", "f16", "bf16", 3),
        # the weights of one decoder layer, hidden 1024 / intermediate 2048 / 4 KV heads, from 32-bit momenta
        _ortho("layer h1024", "1024x1024*2,256x1024*2,2048x1024*2,1024x2048", "f32", "bf16"),
        # four such layers whose consumer keeps 16-bit floats with 11 bits: a result as exact as fp16 holds
        _ortho("layers h1024 to fp16", "1024x1024*8,256x1024*8,2048x1024*8,1024x2048*4", "f16", "f16"),
        # one decoder layer of hidden 2048 / intermediate 8192 / 8 KV heads, 32-bit in and out
        _ortho("layer h2048 in f32", "2048x2048*2,512x2048*2,8192x2048*2,2048x8192", "f32", "f32"),
        # two layers of the same model, bf16 in and out
        _ortho("layers h2048", "2048x2048*4,512x2048*4,8192x2048*4,2048x8192*2", "bf16", "bf16"),
        # the step of a small MLP, one unit a layer, biases under AdamW: latency again
        _mlp("step mlp", "40-128-128-64-32-16", 4, "per unit", "f16", "f16", 1e-3, "rms", True, False),
        # an MLP of odd widths, every parameter sharded along its rows, 32-bit parameters, already reduced gradients
        _mlp("step odd", "333-1000-777-131-5", 5, "per parameter", "bf16", "none", 1e-4, "rows", False, True),
        # the decoder of hidden 1024, 8 layers, 8 replicas in one flat buffer
        _decoder("step 73M", 1024, 2048, 1024, 256, 8, 1024, 8, "global flat", "bf16", "bf16", 1e-4, "rms", True, False),
        # two layers of hidden 2048 under per-parameter shards with 32-bit parameters
        _decoder("step h2048 shards", 2048, 8192, 2048, 512, 2, 8192, 2, "per parameter", "bf16", "none", 1e-4, "rms",
                 True, False),
        # the decoder of hidden 2048, 8 layers, vocabulary 40960: 654M parameters, 2 replicas
        _decoder("step 654M", 2048, 8192, 2048, 512, 8, 40960, 2, "global flat", "bf16", "bf16", 1e-4, "rms", True,
                 False),
    ]


def _spread(rng, lo, hi):
    """A whole number between lo and hi, even over its logarithm."""
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    if rng.random() < 0.5:
        left, mats, shapes = 5e7, 48, []
        for _ in range(_spread(rng, 1, 12)):
            rows, cols = _spread(rng, 1, 8192), _spread(rng, 1, 8192)
            if rng.random() < 0.5:  # widths of real layers are multiples of 64
                rows, cols = max(64, rows // 64 * 64), max(64, cols // 64 * 64)
            if min(rows, cols) > 2048:  # the longer side is the wide one of an MLP, the other the hidden size
                rows, cols = (2048, cols) if rows < cols else (rows, 2048)
            count = _spread(rng, 1, 8)
            if rows * cols * count <= left and count <= mats:
                left, mats = left - rows * cols * count, mats - count
                shapes.append("%dx%d*%d" % (rows, cols, count))
        src, dst = rng.choice(["f32", "bf16", "f16"]), rng.choice(["bf16", "bf16", "f16", "f32"])
        case = _ortho("", ",".join(shapes or ["64x64*1"]), src, dst, rng.choice([0, 0, 1, 8]))
    elif rng.random() < 0.5:
        widths = "-".join(str(_spread(rng, 1, 2048)) for _ in range(rng.randint(2, 7)))
        case = _mlp("", widths, rng.randint(1, 9), rng.choice(sorted(LAYOUTS)), rng.choice(["bf16", "f16"]),
                    rng.choice(["bf16", "f16", "none"]), 1e-4, rng.choice(["rows", "rms"]),
                    rng.random() < 0.7, rng.random() < 0.3)
    else:
        hidden = 64 * _spread(rng, 2, 32)
        case = _decoder("", hidden, 64 * _spread(rng, 2, 128), hidden, 64 * rng.randint(1, 8), rng.randint(1, 4),
                        _spread(rng, 64, 40960), rng.randint(1, 8), rng.choice(sorted(LAYOUTS)),
                        rng.choice(["bf16", "f16"]), rng.choice(["bf16", "f16", "none"]), 1e-4,
                        rng.choice(["rows", "rms"]), rng.random() < 0.7, rng.random() < 0.3)
    del case["name"]
    return case


# ---- sizes and layouts ---------------------------------------------------------------------------------------------

def _shapes(case):
    """(rows, cols) of every matrix of an orthogonalisation."""
    found = []
    for word in case["shapes"].split(","):
        size, _, count = word.partition("*")
        rows, cols = size.split("x")
        found += [(int(rows), int(cols))] * int(count or 1)
    return found


def _parameters(case):
    """Every parameter of the model, in order: (numel, unit, rows (0: a vector), given to Muon, initial deviation)."""
    found = []
    if case["model"] == "mlp":
        widths = [int(w) for w in case["widths"].split("-")]
        for i, (cols, rows) in enumerate(zip(widths, widths[1:])):
            found += [(rows * cols, i, rows, True, 0.02), (rows, i, 0, False, 0.02)]
        return found
    h, inter, q, kv = case["hidden"], case["inter"], case["q"], case["kv"]
    found.append((case["vocab"] * h, 0, case["vocab"], False, 0.02))
    for i in range(case["layers"]):
        for rows, cols in ((q, h), (kv, h), (kv, h), (h, q), (inter, h), (inter, h), (h, inter)):
            found.append((rows * cols, i + 1, rows, True, 0.02))
        found += [(h, i + 1, 0, False, 0.0)] * 2
    last = case["layers"] + 1
    return found + [(h, last, 0, False, 0.0), (case["vocab"] * h, last, case["vocab"], False, 0.02)]


def _layout(case):
    """(offset of every parameter in the padded flat buffer, its whole length).  One flat unit, or one a layer, each
    padded to a multiple of the rank count; or every parameter padded to whole rows a rank."""
    n, at, offsets, unit = case["ranks"], 0, [], 0
    for numel, u, rows, _, _ in _parameters(case):
        if case["layout"] == "per parameter":
            rows = rows or numel
            offsets.append(at)
            at += n * -(-rows // n) * (numel // rows)
        else:
            if case["layout"] == "per unit" and u != unit:
                at = -(-at // n) * n
                unit = u
            offsets.append(at)
            at += numel
    return offsets, -(-at // n) * n


# ---- inputs --------------------------------------------------------------------------------------------------------

def _low_rank(g, rows, cols, device):
    """A gradient's shape: a few strong directions over noise, of about unit deviation."""
    r = min(8, rows, cols)
    strong = torch.randn(rows, r, generator=g, device=device) @ torch.randn(r, cols, generator=g, device=device)
    return torch.randn(rows, cols, generator=g, device=device) + strong * (2.0 / math.sqrt(r))


def _inputs(case, seed):
    device = "cuda"
    g = torch.Generator(device=device).manual_seed(seed)
    if case["op"] == "orthogonalize":
        dt, mats = DTYPES[case["src"]], []
        for rows, cols in _shapes(case):
            wide = torch.zeros(rows, cols + case["gap"], dtype=dt, device=device)
            wide[:, :cols] = (_low_rank(g, rows, cols, device) * 1e-2).to(dt)
            mats.append(wide[:, :cols])
        return {"mats": mats}
    params = _parameters(case)
    offsets, size = _layout(case)
    n, scale = case["ranks"], 1024.0 if case["grad"] == "f16" else 1.0
    master = torch.zeros(size, device=device)
    momentum = torch.zeros(size, device=device)
    square = torch.zeros(size, device=device)
    mean = torch.zeros(size, device=device)
    for (numel, _, rows, muon, deviation), at in zip(params, offsets):
        part = slice(at, at + numel)
        master[part] = torch.randn(numel, generator=g, device=device) * deviation if deviation else 1.0
        if muon:  # the momentum of the steps before, along the gradient's own directions
            strong = _low_rank(g, rows, numel // rows, device).reshape(-1)
            mean[part] = strong * 1e-3
            momentum[part] = strong * 5e-3 + torch.randn(numel, generator=g, device=device) * 1e-3
        else:
            mean[part] = torch.randn(numel, generator=g, device=device) * 1e-3
            momentum[part] = torch.randn(numel, generator=g, device=device) * 3e-4
            square[part] = torch.rand(numel, generator=g, device=device) * 1e-6
    made = {"master": master, "momentum": momentum, "square": square, "loss_scale": scale, "size": size,
            "parameters": params, "offsets": offsets}
    real = torch.zeros(size, dtype=torch.bool, device=device)
    for (numel, *_), at in zip(params, offsets):
        real[at:at + numel] = True
    grads = []
    for _ in range(n):
        noise = torch.randn(size, generator=g, device=device) * 1e-3
        grads.append(((mean + noise) * real * scale).to(DTYPES[case["grad"]]))
    if case["reduced"]:  # backward has reduced them already, into 32-bit shards
        total = grads[0].float()
        for q in grads[1:]:
            total = total + q.float()
        made["sums"], grads = total, None
    made["grads"] = grads
    return made


def prepare(case, seed):
    made = _inputs(case, seed)
    made["case"] = case
    if case["op"] == "orthogonalize":
        made["outs"] = [torch.empty(m.shape, dtype=DTYPES[case["dst"]], device=m.device) for m in made["mats"]]
        if own:  # the batch of addresses and the workspace that a program keeps
            from fsdp_sharded_mixed_amd import zf
            made["batch"] = zf.ortho_batch(made["mats"], made["outs"])
            made["workspace"] = torch.empty(zf.orthogonalize_bytes(made["batch"]), dtype=torch.uint8, device="cuda")
        return made
    size = made["size"]
    made["params"] = made["master"].to(DTYPES[case["param"]]) if case["param"] != "none" else None
    if case["layout"] == "per parameter" and not case["reduced"]:
        made["sums"] = torch.zeros(size, device="cuda")  # the resident 32-bit gradient shards
    made["powers"] = [1.0, 1.0]  # beta1^t, beta2^t of the plain form
    if own:
        from fsdp_sharded_mixed_amd import zf
        segments = [(numel, unit, 0, rows) for numel, unit, rows, _, _ in made["parameters"]]
        made["plan"] = zf.plan_flat(segments, case["ranks"], LAYOUTS[case["layout"]], 2)
        made["muon"] = zf.muon_plan(made["plan"], [i for i, p in enumerate(made["parameters"]) if p[3]])
        made["workspace"] = torch.empty(zf.muon_workspace_bytes(made["muon"]), dtype=torch.uint8, device="cuda")
        made["state"] = torch.empty(zf.state_bytes(), dtype=torch.uint8, device="cuda")
        zf.state_init(made["state"], made["loss_scale"], False)
        made["hp"] = zf.hparams(case["lr"], BETA1, BETA2, EPS, DECAY, MAX_NORM)
        made["mhp"] = zf.muon_hparams(case["lr"], momentum=MOMENTUM, weight_decay=DECAY, nesterov=case["nesterov"],
                                      scale_rule=zf.MUON_SCALE_RMS if case["scale"] == "rms" else zf.MUON_SCALE_ROWS)
    return made


# ---- the plain forms -----------------------------------------------------------------------------------------------

def _newton_schulz(mats):
    """The 32-bit plain form over a stack of equal matrices [k, rows, cols]."""
    a, b, c = NS
    x = mats.float()
    if x.shape[1] > x.shape[2]:
        x = x.transpose(1, 2).contiguous()
    norm = x.double().square().sum((1, 2), keepdim=True).sqrt()
    x = (x.double() / (norm + NS_EPS)).float()
    for _ in range(NS_STEPS):
        gram = torch.bmm(x, x.transpose(1, 2).contiguous())
        x = a * x + torch.bmm(b * gram + c * torch.bmm(gram, gram), x)
    return x.transpose(1, 2) if mats.shape[1] > mats.shape[2] else x


def _stacks(shapes):
    """The places of equal shapes, in order."""
    found = {}
    for i, s in enumerate(shapes):
        found.setdefault(tuple(s), []).append(i)
    return found


def _plain_orthogonalize(s):
    for places in _stacks([m.shape for m in s["mats"]]).values():
        x = _newton_schulz(torch.stack([s["mats"][i] for i in places]))
        for k, i in enumerate(places):
            s["outs"][i].copy_(x[k])
    return s["outs"]


def _update_scale(case, rows, cols):
    return 0.2 * math.sqrt(max(rows, cols)) if case["scale"] == "rms" else math.sqrt(max(1.0, rows / cols))


def _plain_muon(s):
    case, lr = s["case"], s["case"]["lr"]
    total = s.get("sums")
    if not case["reduced"]:
        total = s["grads"][0].float()
        for g in s["grads"][1:]:
            total = total + g.float()
        if "sums" in s:
            s["sums"].copy_(total)
    fine = torch.isfinite(total).all()
    unit = s["loss_scale"] * case["ranks"]
    norm = total.double().square().sum().sqrt() / unit
    gs = (torch.clamp(MAX_NORM / (norm + 1e-6), max=1.0) / unit).float()
    s["powers"] = [s["powers"][0] * BETA1, s["powers"][1] * BETA2]
    g = total * gs
    old = s["master"], s["momentum"], s["square"]
    # AdamW everywhere, Muon's matrices written over it
    m = BETA1 * old[1] + (1.0 - BETA1) * g
    v = BETA2 * old[2] + (1.0 - BETA2) * (g * g)
    w = old[0] * (1.0 - lr * DECAY) - lr * ((m / (1.0 - s["powers"][0])) / ((v / (1.0 - s["powers"][1])).sqrt() + EPS))
    chosen = [(numel // rows, rows, at) for (numel, _, rows, muon, _), at in zip(s["parameters"], s["offsets"]) if muon]
    for (cols, rows), places in _stacks([c[:2] for c in chosen]).items():
        parts = [slice(chosen[i][2], chosen[i][2] + rows * cols) for i in places]
        here = torch.stack([g[p] for p in parts])
        moment = MOMENTUM * torch.stack([old[1][p] for p in parts]) + here
        update = here + MOMENTUM * moment if case["nesterov"] else moment
        update = _newton_schulz(update.view(-1, rows, cols)).reshape(len(places), -1)
        rate = lr * _update_scale(case, rows, cols)
        for k, p in enumerate(parts):
            m[p], v[p] = moment[k], old[2][p]
            w[p] = old[0][p] * (1.0 - lr * DECAY) - rate * update[k]
    for buffer, new in zip(old, (w, m, v)):
        buffer.copy_(torch.where(fine, new, buffer))
    if s["params"] is not None:
        s["params"].copy_(torch.where(fine, s["master"].to(s["params"].dtype), s["params"]))
    return _of_step(s)


def _of_step(s):
    out = {"master": s["master"], "momentum": s["momentum"], "square": s["square"]}
    if s["params"] is not None:
        out["params"] = s["params"]
    if s["case"]["layout"] == "per parameter":
        out["sums"] = s["sums"]
    return out


def run(s):
    case = s["case"]
    if not own:
        return _plain_orthogonalize(s) if case["op"] == "orthogonalize" else _plain_muon(s)
    from fsdp_sharded_mixed_amd import zf
    if case["op"] == "orthogonalize":
        zf.orthogonalize(s["batch"], s["workspace"])
        return s["outs"]
    code = {"f16": zf.F16, "bf16": zf.BF16, "none": zf.BF16}
    zf.muon_step(s["muon"], s["hp"], s["mhp"], code[case["grad"]], code[case["param"]], s["grads"], s["master"],
                 s["momentum"], s["square"], s["params"], s["workspace"], s["state"], grad_shards=s.get("sums"),
                 grads_reduced=case["reduced"])
    return _of_step(s)


# ---- the work ------------------------------------------------------------------------------------------------------

def _ns_flops(rows, cols):
    """Products with a symmetric result count once.  Every step needs three square products besides one; the long side
    enters a Gram product (m^2 n) and an application (2 m^2 n) at least three times in five steps if operands hold 16
    bits, since the Gram matrix squares the condition number: 20 m^3 + 9 m^2 (n - m)."""
    m, n = min(rows, cols), max(rows, cols)
    return 20.0 * m ** 3 + 9.0 * m * m * (n - m)


def work(case):
    if case["op"] == "orthogonalize":
        size = {"f16": 2, "bf16": 2, "f32": 4}
        shapes = _shapes(case)
        return {"bytes": sum(r * c for r, c in shapes) * (size[case["src"]] + size[case["dst"]]),
                "flops": sum(_ns_flops(r, c) for r, c in shapes)}
    total = flops = 0
    for numel, _, rows, muon, _ in _parameters(case):
        total += numel * (4 if case["reduced"] else 2 * case["ranks"])
        total += numel * (16 if muon else 24) + (2 * numel if case["param"] != "none" else 0)
        if case["layout"] == "per parameter" and not case["reduced"]:
            total += 4 * numel
        flops += _ns_flops(rows, numel // rows) if muon else 15 * numel
    return {"bytes": total, "flops": flops}


# ---- the definition in 64 bits -------------------------------------------------------------------------------------

def _polar_64(u):
    """The quintic iteration on one matrix in 64 bits, from the side that is shorter."""
    a, b, c = NS
    u = u / (torch.sqrt((u * u).sum()) + NS_EPS)
    tall = u.shape[0] > u.shape[1]
    for _ in range(NS_STEPS):
        if tall:  # on the right: U (a + b U'U + c (U'U)^2)
            r = u.t().contiguous() @ u
            u = a * u + u @ (b * r + c * (r @ r))
        else:
            r = u @ u.t().contiguous()
            u = a * u + (b * r + c * (r @ r)) @ u
    return u


def exact(case, seed):
    made = _inputs(case, seed)
    if case["op"] == "orthogonalize":
        return [_polar_64(m.double()) for m in made["mats"]]
    lr, n = case["lr"], case["ranks"]
    total = made["sums"].double() if case["reduced"] else sum(g.double() for g in made["grads"])
    norm = torch.linalg.vector_norm(total) / (made["loss_scale"] * n)
    g = total * (torch.clamp(MAX_NORM / (norm + 1e-6), max=1.0) / (made["loss_scale"] * n))
    w, m, v = made["master"].double(), made["momentum"].double(), made["square"].double()
    for (numel, _, rows, muon, _), at in zip(made["parameters"], made["offsets"]):
        p = slice(at, at + numel)
        if muon:
            cols = numel // rows
            m[p] = MOMENTUM * m[p] + g[p]
            u = g[p] + MOMENTUM * m[p] if case["nesterov"] else m[p]
            o = _polar_64(u.view(rows, cols)).reshape(-1)
            w[p] = w[p] - lr * (DECAY * w[p] + _update_scale(case, rows, cols) * o)
        else:
            m[p] = BETA1 * m[p] + (1 - BETA1) * g[p]
            v[p] = BETA2 * v[p] + (1 - BETA2) * g[p] ** 2
            first, second = m[p] / (1 - BETA1), v[p] / (1 - BETA2)
            w[p] = w[p] - lr * (DECAY * w[p] + first / (torch.sqrt(second) + EPS))
    out = {"master": w, "momentum": m, "square": v}
    if case["param"] != "none":
        out["params"] = w
    if case["layout"] == "per parameter":
        out["sums"] = total
    return out
