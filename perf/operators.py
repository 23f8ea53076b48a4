"""The operators on the way from gradients to updated parameters: what is measured.

* ``norm``: the global norm of a list of gradient tensors, each tensor's own norm, and the clipping
  coefficient ``coef = grad_scale * min(1, max_norm / (norm + 1e-6))``.
* ``clip``: the same, then ``out = coef * gradient`` for every tensor, in the output's type.
* ``step``: the same, then one Adam step with decoupled weight decay over every tensor, on ``coef * gradient``.

A case is a list of tensors: one hash table, plane set or nothing (``table`` values) and ``small`` tensors of
0 to ``longest`` values (log-uniform lengths from ``lens_seed``; with ``small`` = 1 it has exactly ``longest``).
The small tensors are views of one buffer, packed end to end (``packed``) as in a communication bucket, or each
on a 64-value boundary.  The plain forms work on whole buffers, whatever the number of tensors; the gaps hold
zeros, which change neither a norm nor an update.
"""
import random

import torch

own = False

TYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
BETAS, EPS, CLIP_EPS = (0.9, 0.99), 1e-15, 1e-6
STEP0 = 100                         # steps already taken
RATES = ((1e-3, 0.0), (1e-3, 1e-2))  # (learning rate, weight decay) of the table and of the small tensors


def _case(name, op, table, small, longest, dtype="f32", out="f32", norm="l2", max_norm=1.0, grad_scale=1.0,
          packed=True, work=True, lens_seed=0):
    return dict(name=name, op=op, table=table, small=small, longest=longest, dtype=dtype, out=out, norm=norm,
                max_norm=max_norm, grad_scale=grad_scale, packed=packed, work=work, lens_seed=lens_seed)


def listed():
    return [
        # the smallest decoder's gradients (4 levels of 4096 entries, 651 weights): latency
        _case("norm_tiny", "norm", 32768, 1, 651),
        # a 16-level fp16 grid of 2^19 entries and its network, fp32 gradients
        _case("norm_sports", "norm", 16777216, 1, 6987),
        # a 2^21-entry grid whose gradients came back in fp16 under a loss scale
        _case("norm_paper_f16", "norm", 134217728, 1, 36920, dtype="f16", grad_scale=1 / 1024),
        # many small tensors of odd lengths, packed end to end: the largest entry of each and of all
        _case("norm_many_max", "norm", 0, 300, 65536, norm="inf", lens_seed=3),
        # the smallest decoder, clipped
        _case("clip_tiny", "clip", 32768, 1, 651),
        # HexPlane planes and network, clipped
        _case("clip_hexplane", "clip", 11483136, 1, 44858),
        # fp16 gradients unscaled and clipped into the fp32 ones that the optimiser takes
        _case("clip_unscale_f16", "clip", 16777216, 40, 20000, dtype="f16", grad_scale=1 / 1024, lens_seed=5),
        # the smallest decoder's whole update
        _case("step_tiny", "step", 32768, 1, 651, work=False),
        # many networks and per-Gaussian parameters, bf16 gradients in one packed bucket
        _case("step_many_bf16", "step", 0, 200, 65536, dtype="bf16", lens_seed=7),
        # the sports decoder's update with its fp16 working copies
        _case("step_sports", "step", 16777216, 1, 6987),
        # the 2^21-entry grid and its four heads
        _case("step_paper", "step", 134217728, 1, 36920),
    ]


def draw(rng):
    op = rng.choice(("norm", "clip", "step"))
    table = rng.choice((0, int(2 ** rng.uniform(8, 26.5)), int(2 ** rng.uniform(8, 26.5))))
    dtype = rng.choice(("f32", "f32", "f16", "bf16"))
    return dict(op=op, table=table, small=int(2 ** rng.uniform(0, 8.5)), longest=int(2 ** rng.uniform(3, 16)),
                dtype=dtype, out=rng.choice(("f32", "bf16" if dtype == "bf16" else "f32")), norm=rng.choice(("l2", "l2", "inf", "l1")),
                max_norm=rng.choice((0.1, 1.0, 10.0, 1e6)), grad_scale=rng.choice((1.0, 0.125, 1 / 1024)),
                packed=rng.random() < 0.5, work=rng.random() < 0.7, lens_seed=rng.randrange(1 << 20))


def _lengths(case):
    if case["small"] == 1:
        return [case["longest"]]
    r = random.Random(case["lens_seed"])
    lens = [int((case["longest"] + 1) ** r.random()) - 1 for _ in range(case["small"])]
    lens[r.randrange(len(lens))] = case["longest"]
    return lens


def _layout(case):
    """(lengths, offsets, values) of the small tensors' buffer."""
    lens, at, offsets = _lengths(case), 0, []
    for n in lens:
        offsets.append(at)
        at += n if case["packed"] else -(-n // 64) * 64
    return lens, offsets, max(at, 1)


def _views(flat, lens, offsets):
    return [flat[o:o + n] for n, o in zip(lens, offsets)]


def _inputs(case, seed):
    """Per buffer: gradient, parameters, m, v and the tensors' places in it, from the seed alone."""
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    lens, offsets, total = _layout(case)
    buffers = [] if not case["table"] else [(case["table"], [case["table"]], [0])]
    buffers.append((total, lens, offsets))
    out = []
    for k, (n, ls, os_) in enumerate(buffers):
        table = bool(case["table"]) and k == 0
        rand = lambda: torch.rand(n, device="cuda", generator=gen)
        # heavy-tailed gradients, a third of a table's entries untouched by the batch
        g = torch.randn(n, device="cuda", generator=gen) * 1e-3 * torch.exp(3.0 * rand())
        if table:
            g *= rand() < 0.67
        live = torch.zeros(n, dtype=torch.bool, device="cuda")
        if case["packed"] or table:
            live[:] = True
        else:
            places = torch.tensor([o for o, l in zip(os_, ls) if l], device="cuda")
            ends = torch.tensor([o + l for o, l in zip(os_, ls) if l], device="cuda")
            mark = torch.zeros(n + 1, dtype=torch.int32, device="cuda")
            mark[places] += 1
            mark[ends] -= 1
            live = mark.cumsum(0)[:n] > 0
        g *= live
        b = dict(g=(g / case["grad_scale"]).to(TYPES[case["dtype"]]), lens=ls, offsets=os_, rate=RATES[0 if table else 1])
        if case["op"] == "step":
            m = torch.randn(n, device="cuda", generator=gen) * 1e-3
            m *= live
            v = (m * m * (1.0 + rand()) + 1e-8) * live
            p = torch.randn(n, device="cuda", generator=gen) * (1e-4 if table else 0.1) * live
            b.update(p=p, m=m, v=v)
        out.append(b)
    return out


def prepare(case, seed):
    buffers = _inputs(case, seed)
    for b in buffers:
        if case["op"] == "step":
            b["w"] = b["p"].to(torch.float16) if case["work"] else None
        if case["op"] == "clip":
            b["out"] = torch.zeros_like(b["g"], dtype=TYPES[case["out"]])
        b["ends"] = torch.tensor([o + n for o, n in zip(b["offsets"], b["lens"])], device="cuda")
        b["starts"] = torch.tensor(b["offsets"], device="cuda")
    state = dict(case=case, buffers=buffers, step=torch.full((), STEP0, dtype=torch.int32, device="cuda"))
    if own:
        from spatiotemporal_neural_field_b200 import spin4d as sp
        every = lambda key: [v for b in buffers for v in _views(b[key], b["lens"], b["offsets"])]
        if case["op"] == "step":
            rates = [b["rate"] for b in buffers for _ in b["lens"]]
            state["adam"] = sp.adam_list(every("p"), every("g"), every("m"), every("v"), lr=[r[0] for r in rates],
                                         weight_decay=[r[1] for r in rates],
                                         params_work=every("w") if case["work"] else None)
        state["list"] = sp.grad_list(every("g"), every("out") if case["op"] == "clip" else None)
        state["control"] = sp.grad_control("cuda", step=STEP0)
        state["norms"] = torch.empty(len(state["list"]), dtype=torch.float32, device="cuda")
        state["workspace"] = torch.empty(sp.grad_norm_workspace(len(state["list"])), dtype=torch.uint8, device="cuda")
    return state


def _tensor_sums(b, kind):
    """Each tensor's sum of squares, of magnitudes, or largest magnitude; squares in 32 bits, sums in 64."""
    g = b["g"].float()
    a = g * g if kind == "l2" else g.abs()
    if len(b["lens"]) == 1:
        return (a.amax() if kind == "inf" else a.sum(dtype=torch.float64)).reshape(1)
    if kind == "inf":
        at = torch.searchsorted(b["ends"], torch.arange(a.numel(), device=a.device), right=True)
        at = at.clamp_(max=len(b["lens"]) - 1)   # what lies between or behind the tensors is zero
        return torch.zeros(len(b["lens"]), device=a.device).scatter_reduce_(0, at, a, "amax")
    run = torch.cat([torch.zeros(1, dtype=torch.float64, device=a.device), torch.cumsum(a, 0, dtype=torch.float64)])
    return run[b["ends"]] - run[b["starts"]]


def _plain_norm(state):
    case = state["case"]
    kind, scale = case["norm"], case["grad_scale"]
    sums = torch.cat([_tensor_sums(b, kind) for b in state["buffers"]])
    total = sums.amax() if kind == "inf" else sums.sum()
    if kind == "l2":
        sums, total = sums.clamp(min=0).sqrt(), total.sqrt()
    norm = scale * total.double()
    coef = scale * (case["max_norm"] / (norm + CLIP_EPS)).clamp(max=1.0)
    state["step"] += torch.isfinite(norm)
    return norm.float(), coef.float(), (scale * sums).float()


def _plain_adam(b, coef, step):
    b1, b2 = BETAS
    lr, decay = b["rate"]
    g = b["g"].float() * coef
    b["m"].mul_(b1).add_(g * (1 - b1))
    b["v"].mul_(b2).add_(g * g * (1 - b2))
    t = step.double()
    mhat = b["m"] * (1 / (1 - b1 ** t)).float()
    vhat = b["v"] * (1 / (1 - b2 ** t)).float()
    b["p"].sub_(lr * mhat / (vhat.sqrt() + EPS) + lr * decay * b["p"])
    if b["w"] is not None:
        b["w"].copy_(b["p"])
    return b


def run(state):
    case, buffers = state["case"], state["buffers"]
    if own:
        from spatiotemporal_neural_field_b200 import spin4d as sp
        ctl, norms = state["control"], state["norms"]
        sp.grad_norm(state["list"], ctl, max_norm=case["max_norm"], norm_type=case["norm"],
                     grad_scale=case["grad_scale"], norms=norms, workspace=state["workspace"])
        out = dict(norm=ctl.norm, coef=ctl.coef, norms=norms, step=ctl.step)
        if case["op"] == "clip":
            sp.clip_grads(state["list"], ctl)
        if case["op"] == "step":
            sp.adam_step_tensors(state["adam"], *BETAS, EPS, control=ctl)
    else:
        norm, coef, norms = _plain_norm(state)
        out = dict(norm=norm, coef=coef, norms=norms, step=state["step"])
        if case["op"] == "clip":
            [b["out"].copy_(b["g"].float() * coef) for b in buffers]
        if case["op"] == "step":
            [_plain_adam(b, coef, state["step"]) for b in buffers]
    if case["op"] == "clip":
        out["out"] = [b["out"] for b in buffers]
    if case["op"] == "step":
        out["params"] = [[b["p"], b["m"], b["v"]] for b in buffers]
        out["work"] = [b["w"] for b in buffers if b["w"] is not None]
    return out


def work(case):
    lens, _, _ = _layout(case)
    n = case["table"] + sum(lens)
    g = 4 if case["dtype"] == "f32" else 2
    if case["op"] == "norm":
        return {"bytes": n * g + 4 * len(lens), "flops": 2 * n}
    if case["op"] == "clip":
        return {"bytes": n * (g + (4 if case["out"] == "f32" else 2)), "flops": 3 * n}
    return {"bytes": n * (g + 24 + (2 if case["work"] else 0)), "flops": 18 * n}


def exact(case, seed):
    buffers = _inputs(case, seed)
    scale, kind = case["grad_scale"], case["norm"]
    sums, total = [], 0.0
    for b in buffers:
        for v in _views(b["g"], b["lens"], b["offsets"]):
            x = v.double().abs()
            one = 0.0 if not x.numel() else float({"l2": x.pow(2).sum, "l1": x.sum, "inf": x.max}[kind]())
            total = max(total, one) if kind == "inf" else total + one
            sums.append(one ** 0.5 if kind == "l2" else one)
    norm = scale * (total ** 0.5 if kind == "l2" else total)
    coef = scale * min(1.0, case["max_norm"] / (norm + CLIP_EPS))
    f64 = lambda x: torch.tensor(x, dtype=torch.float64)
    out = dict(norm=f64(norm), coef=f64(coef), norms=f64(sums) * scale, step=torch.tensor(STEP0 + 1))
    if case["op"] == "clip":
        out["out"] = [b["g"].double() * coef for b in buffers]
    if case["op"] == "step":
        b1, b2 = BETAS
        out["params"], out["work"] = [], []
        for b in buffers:
            g = b["g"].double() * coef
            m = b1 * b["m"].double() + (1 - b1) * g
            v = b2 * b["v"].double() + (1 - b2) * g.pow(2)
            p, (lr, decay) = b["p"].double(), b["rate"]
            p = p * (1 - lr * decay) - lr * (m / (1 - b1 ** (STEP0 + 1))) / ((v / (1 - b2 ** (STEP0 + 1))).sqrt() + EPS)
            out["params"].append([p, m, v])
            if case["work"]:
                out["work"].append(p)
    return out
