"""What is measured of the operators around a fine-tuning step's dense layers: the token embedding with its
gradient, the queries' and keys' norm and position rotation with theirs, and distillation from a teacher's top
logits with its gradient.

`listed` and `draw` give cases, `prepare` makes a case's inputs on the GPU from a seed, `run` makes one pass: in
elementary torch operations where `own` is false, through the framework's calls where it is true.  `exact` is the
same from the definitions in 64 bits, and `work` what a pass cannot do without."""
import math

import torch

own = False

BF16 = torch.bfloat16
F32 = torch.float32
F64 = torch.float64
IGNORE = -100


def listed():
    return [
        # One decoding step of eight sequences: the smallest lookup, all latency.
        {"name": "embed_decode", "op": "embed", "pass": "forward", "N": 8, "V": 128256, "d": 4096, "scale": 1.0,
         "zipf": True, "pad": 0.0, "dtype": "bf16"},
        # A packed batch of 32768 tokens of a 2048-wide model whose embeddings are scaled by sqrt(width).
        {"name": "embed_packed", "op": "embed", "pass": "forward", "N": 32768, "V": 32000, "d": 2048,
         "scale": 45.25, "zipf": True, "pad": 0.0, "dtype": "bf16"},
        # The gradient of an 8B model's embedding for one 4096-token step: mostly rows that no token touched.
        {"name": "embed_grad", "op": "embed", "pass": "backward", "N": 4096, "V": 128256, "d": 4096, "scale": 1.0,
         "zipf": True, "pad": 0.0, "dtype": "bf16"},
        # A padded batch under a 256K vocabulary, gradient kept in 32 bits: one id takes a third of the tokens.
        {"name": "embed_grad_padded", "op": "embed", "pass": "backward", "N": 16001, "V": 256000, "d": 2048,
         "scale": 45.25, "zipf": True, "pad": 0.33, "dtype": "fp32"},
        # One decoding step of eight sequences at far positions: normed and rotated queries and keys.
        {"name": "qk_decode", "op": "qk", "pass": "forward", "B": 8, "S": 1, "Hq": 32, "Hk": 8, "D": 128, "rot": 128,
         "norm": True, "interleaved": False, "layout": "bshd", "P": 131072},
        # A 4096-token training step of an 8B model's attention, queries and keys as parts of one projection.
        {"name": "qk_train", "op": "qk", "pass": "both", "B": 1, "S": 4096, "Hq": 32, "Hk": 8, "D": 128, "rot": 128,
         "norm": True, "interleaved": False, "layout": "packed", "P": 8192},
        # 32768 packed tokens of a 1.1B model without norms of queries and keys: the rotation alone.
        {"name": "rope_train_long", "op": "qk", "pass": "both", "B": 16, "S": 2048, "Hq": 32, "Hk": 4, "D": 64,
         "rot": 64, "norm": False, "interleaved": False, "layout": "bshd", "P": 4096},
        # Heads-first tensors of odd sizes, half of each head rotated in neighbouring pairs.
        {"name": "qk_partial_odd", "op": "qk", "pass": "both", "B": 3, "S": 1237, "Hq": 14, "Hk": 2, "D": 96,
         "rot": 48, "norm": True, "interleaved": True, "layout": "bhsd", "P": 2048},
        # A handful of rows over a small odd vocabulary in padded rows.
        {"name": "distill_tiny", "op": "distill", "pass": "loss_grad", "N": 37, "V": 1003, "K": 8, "tau": 1.0,
         "scale": 1.0, "cap": 0.0, "values": "fp32", "ids": "int64"},
        # A training step of an 8B model from stored top-64 logits: loss and gradient.
        {"name": "distill_train", "op": "distill", "pass": "loss_grad", "N": 4096, "V": 128256, "K": 64, "tau": 2.0,
         "scale": 1.0, "cap": 0.0, "values": "bf16", "ids": "int32"},
        # A 256K vocabulary with softcapped logits.
        {"name": "distill_softcap", "op": "distill", "pass": "loss_grad", "N": 1024, "V": 256000, "K": 128,
         "tau": 1.0, "scale": 1.0, "cap": 30.0, "values": "bf16", "ids": "int64"},
        # Validation: the loss of each row, no gradient.
        {"name": "distill_eval", "op": "distill", "pass": "rows", "N": 2047, "V": 128256, "K": 20, "tau": 1.0,
         "scale": 1.0, "cap": 0.0, "values": "fp32", "ids": "int64"},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(("embed", "qk", "distill"))
    if op == "embed":
        back = rng.random() < 0.6
        V = _log(rng, 500, 256000)
        d = 8 * _log(rng, 8, 1024)
        while back and V * d > 450_000_000:
            V = V // 2 + 1
        N = min(_log(rng, 1, 65536), (150_000_000 if back else 500_000_000) // d)
        return {"op": "embed", "pass": "backward" if back else "forward", "N": N, "V": V, "d": d,
                "scale": rng.choice((1.0, round(math.sqrt(d), 3))), "zipf": rng.random() < 0.8,
                "pad": rng.choice((0.0, round(rng.uniform(0.05, 0.6), 3))),
                "dtype": rng.choice(("bf16", "fp32")) if back else "bf16"}
    if op == "qk":
        D = rng.choice((32, 64, 80, 96, 128, 128, 192, 256))
        Hk = rng.choice((1, 2, 4, 8, 16))
        Hq = Hk * rng.choice((1, 2, 4, 7, 8))
        B = rng.randint(1, 8)
        S = max(1, min(_log(rng, 1, 16384), 150_000_000 // (B * (Hq + Hk) * D)))
        return {"op": "qk", "pass": rng.choice(("forward", "both", "both")), "B": B, "S": S, "Hq": Hq, "Hk": Hk, "D": D,
                "rot": rng.choice((D, D, 16 * rng.randint(1, D // 16))), "norm": rng.random() < 0.7,
                "interleaved": rng.random() < 0.4, "layout": rng.choice(("bshd", "packed", "bhsd")),
                "P": S + _log(rng, 1, 100000)}
    V = _log(rng, 100, 256000)
    return {"op": "distill", "pass": rng.choice(("loss_grad", "loss_grad", "rows")),
            "N": max(1, min(_log(rng, 1, 8192), 500_000_000 // V)), "V": V, "K": min(V // 2, _log(rng, 1, 512)),
            "tau": rng.choice((1.0, 2.0, round(rng.uniform(0.5, 4.0), 2))),
            "scale": rng.choice((1.0, 0.0625)), "cap": rng.choice((0.0, 0.0, 30.0, 50.0)),
            "values": rng.choice(("bf16", "fp32")), "ids": rng.choice(("int32", "int64"))}


def work(case):
    if case["op"] == "embed":
        N, V, d = case["N"], case["V"], case["d"]
        if case["pass"] == "forward":  # a row that several tokens share is read once at best
            return {"bytes": N * 8 + 2 * min(N, V) * d + 2 * N * d, "flops": N * d}
        return {"bytes": N * 8 + 2 * N * d + (2 if case["dtype"] == "bf16" else 4) * V * d, "flops": 2 * N * d}
    if case["op"] == "qk":
        T, H, D = case["B"] * case["S"], case["Hq"] + case["Hk"], case["D"]
        n = T * H * D
        table = 4 * min(T, case["P"]) * case["rot"] + 8 * T
        b, f = 4 * n + table, (7 if case["norm"] else 3) * n
        if case["pass"] == "both":
            b += (6 if case["norm"] else 4) * n + table
            f += (14 if case["norm"] else 3) * n
        return {"bytes": b, "flops": f}
    N, V, K = case["N"], case["V"], case["K"]
    pairs = N * K * ((2 if case["values"] == "bf16" else 4) + (4 if case["ids"] == "int32" else 8)) + 8 * N
    if case["pass"] == "rows":
        return {"bytes": 2 * N * V + pairs + 4 * N, "flops": 4 * N * V}
    return {"bytes": 4 * N * V + pairs, "flops": 8 * N * V}


# --------------------------------------------------------------------------- inputs


def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _ids(case, g):
    """Token ids as text has them: a few ids take many tokens, most ids none; `pad` of the tokens are id 0."""
    N, V = case["N"], case["V"]
    u = torch.rand(N, device="cuda", generator=g, dtype=F64)
    if case["zipf"]:
        rank = torch.exp(u * math.log(V + 1.0)).floor().long() - 1
        ids = (rank.clamp(0, V - 1) * 7919 + 13) % V  # frequent ids lie apart, as in a real vocabulary
    else:
        ids = (u * V).long().clamp(max=V - 1)
    if case["pad"]:
        ids = torch.where(torch.rand(N, device="cuda", generator=g) < case["pad"], torch.zeros_like(ids), ids)
    return ids


def prepare(case, seed):
    g = _gen(seed)
    if case["op"] == "embed":
        state = {"case": case, "ids": _ids(case, g)}
        if case["pass"] == "forward":
            state["E"] = torch.randn(case["V"], case["d"], device="cuda", generator=g, dtype=BF16) * 0.02
        else:
            state["dOut"] = torch.randn(case["N"], case["d"], device="cuda", generator=g, dtype=BF16) * 0.01
        return state
    if case["op"] == "qk":
        B, S, Hq, Hk, D, P, rot = (case[x] for x in ("B", "S", "Hq", "Hk", "D", "P", "rot"))

        def heads():
            if case["layout"] == "packed":  # parts of one projection's output, values behind them
                y = torch.randn(B, S, (Hq + 2 * Hk) * D, device="cuda", generator=g, dtype=BF16)
                return (y[..., :Hq * D].view(B, S, Hq, D), y[..., Hq * D:(Hq + Hk) * D].view(B, S, Hk, D))
            if case["layout"] == "bhsd":
                return tuple(torch.randn(B, h, S, D, device="cuda", generator=g, dtype=BF16).transpose(1, 2)
                             for h in (Hq, Hk))
            return tuple(torch.randn(B, S, h, D, device="cuda", generator=g, dtype=BF16) for h in (Hq, Hk))

        start = torch.randint(0, P - S + 1, (B, 1), device="cuda", generator=g)
        angle = (torch.arange(P, device="cuda", dtype=F64)[:, None]
                 * 500000.0 ** (-torch.arange(0, rot, 2, device="cuda", dtype=F64) / rot))
        state = {"case": case, "positions": start + torch.arange(S, device="cuda"), "cos": angle.cos().float(),
                 "sin": angle.sin().float(), "eps": 1e-6, "q_gain": None, "k_gain": None}
        state["q"], state["k"] = heads()
        if case["norm"]:
            state["q_gain"], state["k_gain"] = (
                (0.5 + torch.rand(D, device="cuda", generator=g)).to(BF16) for _ in range(2))
        if case["pass"] == "both":  # what attention's backward hands over: its own dense tensors
            state["dq"] = torch.randn(B, S, Hq, D, device="cuda", generator=g, dtype=BF16)
            state["dk"] = torch.randn(B, S, Hk, D, device="cuda", generator=g, dtype=BF16)
        return state
    N, V, K = case["N"], case["V"], case["K"]
    z = torch.zeros(N, (V + 7) // 8 * 8, device="cuda", dtype=BF16)[:, :V]
    z.normal_(0.0, 2.0, generator=g)
    # K different ids a row, the teacher's values in falling order, a student that has come near them.
    ids = torch.arange(K, device="cuda") * V // K + (torch.rand(N, K, device="cuda", generator=g) * (V // K)).long()
    ids = ids.gather(1, torch.rand(N, K, device="cuda", generator=g).argsort(1))
    values = (torch.randn(N, K, device="cuda", generator=g) * 2.0 + 8.0).sort(1, descending=True).values
    near = values + torch.randn(N, K, device="cuda", generator=g)
    z.scatter_(1, ids, near.to(BF16))
    if case["scale"] != 1.0:
        z /= case["scale"]
    if K > 1:  # a tenth of the rows keep fewer entries: the rest is -1
        keep = torch.where(torch.rand(N, 1, device="cuda", generator=g) < 0.1,
                           torch.randint(1, K, (N, 1), device="cuda", generator=g), K)
        ids = torch.where(torch.arange(K, device="cuda") < keep, ids, -1)
    labels = torch.randint(0, V, (N,), device="cuda", generator=g)
    labels = torch.where(torch.rand(N, device="cuda", generator=g) < 0.03, IGNORE, labels)
    return {"case": case, "logits": z, "labels": labels,
            "values": values.to(BF16 if case["values"] == "bf16" else F32),
            "ids": ids.to(torch.int32 if case["ids"] == "int32" else torch.int64)}


# --------------------------------------------------------------------------- one pass


def run(state):
    op = state["case"]["op"]
    if op == "embed":
        return _run_embed(state)
    if op == "qk":
        return _run_qk(state)
    return _run_distill(state)


def _run_embed(state):
    case, ids = state["case"], state["ids"]
    dtype = BF16 if case["dtype"] == "bf16" else F32
    if own:
        from lora_fine_tuning_mlp_b200 import api
        if case["pass"] == "forward":
            return api.embedding_forward(ids, state["E"], scale=case["scale"])
        return api.embedding_backward(state["dOut"], ids, case["V"], scale=case["scale"], dtype=dtype)
    if case["pass"] == "forward":
        return (state["E"][ids].float() * case["scale"]).to(BF16)
    dE = torch.zeros(case["V"], case["d"], device="cuda", dtype=F32)
    return dE.index_add_(0, ids, state["dOut"].float()).mul_(case["scale"]).to(dtype)


def _angles(state):
    cos, sin = state["cos"][state["positions"]], state["sin"][state["positions"]]
    return cos[:, :, None, :], sin[:, :, None, :]


def _rotate(x, cos, sin, interleaved):
    rot = 2 * cos.shape[-1]
    if interleaved:
        a, b = x[..., 0:rot:2], x[..., 1:rot:2]
        y = torch.stack((a * cos - b * sin, b * cos + a * sin), -1).flatten(-2)
    else:
        a, b = x[..., :rot // 2], x[..., rot // 2:rot]
        y = torch.cat((a * cos - b * sin, b * cos + a * sin), -1)
    return torch.cat((y, x[..., rot:]), -1)


def _plain_forward(x, gain, eps, cos, sin, interleaved):
    y = x.float()
    if gain is not None:
        y = y * (y.square().mean(-1, keepdim=True) + eps).rsqrt() * gain.float()
    return _rotate(y, cos, sin, interleaved).to(BF16)


def _plain_backward(x, gain, eps, cos, sin, interleaved, dout):
    dy = _rotate(dout.float(), cos, -sin, interleaved)
    if gain is None:
        return dy.to(BF16), None
    r = (x.float().square().mean(-1, keepdim=True) + eps).rsqrt()
    n = x.float() * r
    dn = dy * gain.float()
    return (r * (dn - n * (dn * n).mean(-1, keepdim=True))).to(BF16), (dy * n).sum((0, 1, 2))


def _run_qk(state):
    case, q, k = state["case"], state["q"], state["k"]
    if own:
        from lora_fine_tuning_mlp_b200 import api
        kw = {"positions": state["positions"], "q_gain": state["q_gain"], "k_gain": state["k_gain"],
              "eps": state["eps"], "interleaved": case["interleaved"]}
        qo, ko = api.qk_norm_rope_forward(q, k, state["cos"], state["sin"], **kw)
        if case["pass"] == "forward":
            return [qo, ko]
        return [qo, ko, *api.qk_norm_rope_backward(q, k, state["cos"], state["sin"], state["dq"], state["dk"], **kw)]
    cos, sin = _angles(state)
    common = (state["eps"], cos, sin, case["interleaved"])
    qo, ko = _plain_forward(q, state["q_gain"], *common), _plain_forward(k, state["k_gain"], *common)
    if case["pass"] == "forward":
        return [qo, ko]
    dq, dgq = _plain_backward(q, state["q_gain"], *common, state["dq"])
    dk, dgk = _plain_backward(k, state["k_gain"], *common, state["dk"])
    return [qo, ko, dq, dk, dgq, dgk]


def _run_distill(state):
    case, z = state["case"], state["logits"]
    tau, scale, cap = case["tau"], case["scale"], case["cap"]
    if own:
        from lora_fine_tuning_mlp_b200 import api
        kw = {"labels": state["labels"], "temperature": tau, "logit_scale": scale, "softcap": cap,
              "ignore_index": IGNORE}
        if case["pass"] == "rows":
            return api.distill_forward(z, state["values"], state["ids"], **kw)
        out, dz = api.distill_loss(z, state["values"], state["ids"], reduction="mean", **kw)
        return [out[0], dz]
    t = z.float() * scale
    if cap > 0.0:
        t = cap * torch.tanh(t / cap)
    x = t / tau
    x = x - x.max(1, keepdim=True).values
    x = x - x.exp().sum(1, keepdim=True).log()  # log-probabilities of the student
    there = state["ids"] >= 0
    ids = state["ids"].long().clamp(min=0)
    a = torch.where(there, state["values"].float() / tau, -math.inf)
    a = a - a.max(1, keepdim=True).values
    p = a.exp()
    total = p.sum(1, keepdim=True)
    p, logp = p / total, a - total.log()
    part = (state["labels"] != IGNORE).float()
    rows = tau * tau * part * torch.where(there, p * (logp - x.gather(1, ids)), 0.0).sum(1)
    if case["pass"] == "rows":
        return rows
    count = part.sum().clamp(min=1.0)
    dx = x.exp().scatter_add(1, ids, torch.where(there, -p, 0.0))
    dz = dx * (part * (tau * scale) / count)[:, None]
    if cap > 0.0:
        dz = dz * (1.0 - (t / cap).square())
    return [rows.sum() / count, dz.to(BF16)]


# --------------------------------------------------------------------------- from the definitions, in 64 bits


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "embed":
        if case["pass"] == "forward":
            return s["E"].double().index_select(0, s["ids"]) * case["scale"]
        if case["V"] * case["d"] > 600_000_000:
            return None
        order = s["ids"].argsort(stable=True)
        rows, counts = s["ids"][order].unique_consecutive(return_counts=True)
        ends = counts.cumsum(0)
        dE = torch.zeros(case["V"], case["d"], device="cuda", dtype=F64)
        for c in range(0, case["d"], 512):  # sums of a run of equal ids are differences of running sums
            run_sum = torch.cat((torch.zeros_like(s["dOut"][:1, c:c + 512], dtype=F64),
                                 s["dOut"][order, c:c + 512].double().cumsum(0)))
            dE[rows, c:c + 512] = (run_sum[ends] - run_sum[ends - counts]) * case["scale"]
        return dE
    if case["op"] == "qk":
        found = []
        leaves = []
        phase = torch.complex(s["cos"].double(), s["sin"].double())[s["positions"]][:, :, None, :]
        rot = case["rot"]
        for x, gain in ((s["q"], s["q_gain"]), (s["k"], s["k_gain"])):
            x = x.double().contiguous().requires_grad_(True)
            y = x
            if gain is not None:
                gain = gain.double().requires_grad_(True)
                y = x / ((x * x).sum(-1, keepdim=True) / case["D"] + s["eps"]).sqrt() * gain
            head = y[..., :rot]
            if case["interleaved"]:
                turned = torch.view_as_real(torch.view_as_complex(head.unflatten(-1, (rot // 2, 2)).contiguous())
                                            * phase).flatten(-2)
            else:
                turned = torch.complex(head[..., :rot // 2], head[..., rot // 2:]) * phase
                turned = torch.cat((turned.real, turned.imag), -1)
            found.append(torch.cat((turned, y[..., rot:]), -1))
            leaves.append((x, gain))
        outs = [f.detach() for f in found]
        if case["pass"] == "forward":
            return outs
        dx, dgain = [], []
        for f, d, (x, gain) in zip(found, (s["dq"], s["dk"]), leaves):
            got = torch.autograd.grad(f, [x] if gain is None else [x, gain], d.double())
            dx.append(got[0])
            dgain.append(None if gain is None else got[1])
        return outs + dx + dgain
    N, V, tau = case["N"], case["V"], case["tau"]
    if N * V > 600_000_000:
        return None
    taking_part = s["labels"] != IGNORE
    count = max(1, int(taking_part.sum()))
    rows = torch.zeros(N, device="cuda", dtype=F64)
    dz = None if case["pass"] == "rows" else torch.zeros(N, V, device="cuda", dtype=F64)
    step = max(1, 40_000_000 // V)
    for r in range(0, N, step):
        at = slice(r, min(N, r + step))
        z = s["logits"][at].double()
        t = z * case["scale"]
        slope = torch.full_like(t, case["scale"])
        if case["cap"] > 0.0:
            slope = case["scale"] / torch.cosh(t / case["cap"]) ** 2
            t = case["cap"] * torch.tanh(t / case["cap"])
        teacher = torch.zeros_like(t)
        ids, there = s["ids"][at].long(), s["ids"][at] >= 0
        a = torch.softmax(torch.where(there, s["values"][at].double() / tau, -math.inf), 1)
        teacher.scatter_add_(1, ids.clamp(min=0), torch.where(there, a, 0.0))
        student = torch.log_softmax(t / tau, 1)
        kl = (torch.special.xlogy(a, a).sum(1) - (teacher * student).sum(1)) * tau * tau
        rows[at] = torch.where(taking_part[at], kl, 0.0)
        if dz is not None:
            dz[at] = torch.where(taking_part[at, None], (student.exp() - teacher) * slope * (tau / count), 0.0)
    return rows if dz is None else [rows.sum() / count, dz]
