"""The training operators: learned node embeddings (lookup and gradient), the
softmax cross-entropy loss with its gradient, and the orthogonalised (Muon)
weight update, as cases with their inputs, their plain form in torch and the
calls a user of the package makes.

A case is a dict of plain values; "op" names the operator:
  embed_fwd  out[i] = scale * table[ids[i]] (a zero row for ids[i] = -1)
  embed_bwd  the table's gradient: per distinct id the sum of its rows of g,
             as the sorted distinct ids with one row each ("rows"), as the
             whole table ("dense") or added into given rows ("add")
  xent       loss per row, its mean over the labelled rows, and the gradient
  orth       orthogonalisation of a matrix by Newton-Schulz products
  muon       one Muon step: momentum, orthogonalisation, weight update
"""
import math

import torch

own = False

COEF = (3.4445, -4.7750, 2.0315)  # the quintic of the Muon optimiser
DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16}


def listed():
    return [
        # the input nodes of one small mini-batch (256 seeds, two hops): latency counts
        dict(name="embed_fwd_tiny", op="embed_fwd", n=4999, dim=64, n_rows=10000, skew=False, dtype="f32",
             dtype_out="f32"),
        # the input nodes of a three-hop batch of 1024 seeds, from a table past 2^31 elements
        dict(name="embed_fwd_batch", op="embed_fwd", n=600001, dim=128, n_rows=20000000, skew=False, dtype="f32",
             dtype_out="f32"),
        # gradient of a small, wholly resident table
        dict(name="embed_bwd_tiny", op="embed_bwd", n=4999, dim=64, n_rows=10000, skew=False, dtype="f32",
             dtype_out="f32", mode="dense"),
        # a super-batch of 8: its mini-batches repeat each other's nodes, hot ones most; a sparse gradient of a large table
        dict(name="embed_bwd_super", op="embed_bwd", n=800003, dim=256, n_rows=10000000, skew=True, dtype="f32",
             dtype_out="f32", mode="rows"),
        # tokens with a power law over a vocabulary: wide bf16 rows, a few ids with a large share of all positions
        dict(name="embed_bwd_tokens", op="embed_bwd", n=65536, dim=1024, n_rows=50001, skew=True, dtype="bf16",
             dtype_out="bf16", mode="dense"),
        # the loss of a small batch over as many classes as the hidden width
        dict(name="xent_small", op="xent", n=256, classes=128, dtype="f32", masked=False),
        # a few rows over a very long axis
        dict(name="xent_long", op="xent", n=5, classes=131072, dtype="f32", masked=True),
        # a large batch over an odd number of classes (rows start at any 2-byte address)
        dict(name="xent_large", op="xent", n=4096, classes=50257, dtype="bf16", masked=False),
        # one layer's weights of the 100-feature workload (128 x 2*100)
        dict(name="muon_layer", op="muon", count=1, rows=128, cols=200, dtype="f32", nesterov=True),
        # the first layer of the 1024-feature bf16 workload (128 x 2*1024)
        dict(name="muon_wide", op="muon", count=1, rows=128, cols=2048, dtype="bf16", nesterov=True),
        # an odd, tall matrix in bf16
        dict(name="orth_tall", op="orth", count=1, rows=1001, cols=603, dtype="bf16"),
        # a large layer, bound by its matrix products
        dict(name="orth_large", op="orth", count=1, rows=1024, cols=4096, dtype="f32"),
    ]


def _log_int(rng, lo, hi):
    v = int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))
    v = min(hi, max(lo, v))
    return v + 1 if v == 3072 else v


def draw(rng):
    op = rng.choice(["embed_fwd", "embed_bwd", "embed_bwd", "xent", "xent", "orth", "muon"])
    f = rng.choice(["f32", "bf16"])
    if op in ("embed_fwd", "embed_bwd"):
        dim = rng.choice([64, 100, 128, 256, 1024, _log_int(rng, 1, 1024)])
        n = _log_int(rng, 1, min(800000, 100000000 // dim))
        case = dict(op=op, n=n, dim=dim, skew=rng.random() < 0.6, dtype=f, dtype_out=rng.choice(["f32", "bf16"]))
        if op == "embed_bwd":
            case["mode"] = rng.choice(["rows", "dense", "add"])
        most = 20000000 if op == "embed_fwd" or case["mode"] == "rows" else 50000000 // dim  # a dense gradient costs every row
        case["n_rows"] = _log_int(rng, 100, min(20000000, most, 2500000000 // dim))
        return case
    if op == "xent":
        classes = _log_int(rng, 2, 131072)
        return dict(op=op, n=_log_int(rng, 1, max(1, min(65536, 100000000 // classes))), classes=classes, dtype=f,
                    masked=rng.random() < 0.3)
    if rng.random() < 0.6:  # the hidden width of the package's layers
        rows, cols = 128, rng.choice([128, 200, 256, 512, 2048, _log_int(rng, 16, 2048)])
    else:
        rows, cols = _log_int(rng, 16, 1024), _log_int(rng, 16, 4096)
    if rng.random() < 0.2:
        rows, cols = cols, rows
    case = dict(op=op, count=rng.choice([1, 1, 2, 3]) if rows * cols <= 1000000 else 1, rows=rows, cols=cols, dtype=f)
    if op == "muon":
        case["nesterov"] = rng.random() < 0.7
    return case


# ------------------------------------------------------------------- inputs
def _generator(seed, salt):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed * 1000003 + salt)
    return g


def _ids(case, g):
    """int32 ids, 1 % of them -1 (padding); with skew, log-uniform (the
    frequency of id v falls as 1 / (v + 1)), else uniform."""
    n, n_rows = case["n"], case["n_rows"]
    u = torch.rand(n, generator=g, device="cuda", dtype=torch.float64)
    v = torch.exp(u * math.log(n_rows + 1)) - 1 if case["skew"] else u * n_rows
    v = v.to(torch.int64).clamp_(0, n_rows - 1).to(torch.int32)
    pad = torch.rand(n, generator=g, device="cuda") < 0.01
    return torch.where(pad, torch.full_like(v, -1), v)


def _gradient(case, g, salt):
    """count x rows x cols fp32: a few strong directions over noise, as
    weight gradients have."""
    k, r, c = case["count"], case["rows"], case["cols"]
    rank = max(1, min(r, c) // 16)
    left = torch.randn(k, r, rank, generator=g, device="cuda")
    right = torch.randn(k, rank, c, generator=g, device="cuda")
    decay = torch.exp(-4.0 * torch.arange(rank, device="cuda") / rank)
    return 1e-3 * ((left * decay) @ right / math.sqrt(rank) + torch.randn(k, r, c, generator=g, device="cuda"))


def _inputs(case, seed):
    op = case["op"]
    dt = DTYPES[case["dtype"]]
    if op == "embed_fwd":
        g = _generator(seed, 1)
        table = torch.empty(case["n_rows"], case["dim"], dtype=dt, device="cuda").normal_(generator=g)
        return dict(table=table, ids=_ids(case, g), scale=math.sqrt(case["dim"]))
    if op == "embed_bwd":
        g = _generator(seed, 2)
        ids = _ids(case, g)
        out = dict(ids=ids, scale=math.sqrt(case["dim"]),
                   g=(1e-3 * torch.randn(case["n"], case["dim"], generator=g, device="cuda")).to(dt))
        if case["mode"] == "add":
            out["base"] = torch.empty(case["n_rows"], case["dim"], dtype=DTYPES[case["dtype_out"]],
                                      device="cuda").normal_(generator=g)
        return out
    if op == "xent":
        g = _generator(seed, 3)
        n, c = case["n"], case["classes"]
        labels = torch.randint(0, c, (n,), generator=g, device="cuda", dtype=torch.int32)
        x = 2 * torch.randn(n, c, generator=g, device="cuda")
        if case["masked"]:  # a tenth of the classes not to be answered with
            off = torch.rand(n, c, generator=g, device="cuda") < 0.1
            off.scatter_(1, labels.long()[:, None], False)
            x.masked_fill_(off, float("-inf"))
        x.scatter_add_(1, labels.long()[:, None], torch.full((n, 1), 3.0, device="cuda"))
        ignored = torch.rand(n, generator=g, device="cuda") < 0.02
        return dict(logits=x.to(dt), labels=torch.where(ignored, torch.full_like(labels, -1), labels))
    g = _generator(seed, 4)
    grad = _gradient(case, g, 0)
    if op == "orth":
        return dict(g=grad.to(dt))
    w = (torch.randn(grad.shape, generator=g, device="cuda") / math.sqrt(case["cols"])).to(dt)
    return dict(w=w, g=grad, m=_gradient(case, g, 1), lr=0.02, mu=0.95, wd=0.01,
                scale=math.sqrt(max(1.0, case["rows"] / case["cols"])))


def prepare(case, seed):
    state = dict(case=case, **_inputs(case, seed))
    if not own:
        return state
    from sampling_gnn_mini_gb300 import binding as sg
    op = case["op"]
    state["sg"] = sg
    if op == "embed_fwd":
        state["out"] = torch.empty(case["n"], case["dim"], dtype=DTYPES[case["dtype_out"]], device="cuda")
    elif op == "embed_bwd":
        mode = {"rows": sg.SG_GRAD_ROWS, "dense": sg.SG_GRAD_DENSE, "add": sg.SG_GRAD_ADD}[case["mode"]]
        state["mode"] = mode
        state["ws"] = sg.aligned_workspace(sg.sg_embed_bwd_workspace(case["n"], case["n_rows"], case["dim"], mode))
        if mode == sg.SG_GRAD_ROWS:  # entries past the count of distinct ids are left as they are
            state["rows"] = torch.full((case["n"],), -1, dtype=torch.int32, device="cuda")
            state["count"] = torch.zeros(1, dtype=torch.int32, device="cuda")
        shape = (case["n"] if mode == sg.SG_GRAD_ROWS else case["n_rows"], case["dim"])
        state["grad"] = torch.zeros(shape, dtype=DTYPES[case["dtype_out"]], device="cuda")
    elif op == "xent":
        state["loss"] = torch.empty(case["n"], device="cuda")
        state["total"] = torch.empty(2, device="cuda")
        state["grad"] = torch.empty_like(state["logits"])
        state["ws"] = sg.aligned_workspace(sg.sg_xent_workspace(case["n"], case["classes"]))
    else:
        state["ws"] = sg.aligned_workspace(sg.sg_orthogonalise_workspace(case["count"], case["rows"], case["cols"]))
        if op == "orth":
            state["out"] = torch.empty_like(state["g"])
        else:
            state["w_out"], state["m_out"] = torch.empty_like(state["w"]), torch.empty_like(state["m"])
    return state


# --------------------------------------------------------------------- run
def run(state):
    return _run_own(state) if own else _run_plain(state)


def _run_own(s):
    sg, case = s["sg"], s["case"]
    op = case["op"]
    if op == "embed_fwd":
        sg.sg_embed_fwd(s["table"], s["ids"], case["n"], None, s["scale"], s["out"])
        return s["out"]
    if op == "embed_bwd":
        if case["mode"] == "rows":
            sg.sg_embed_bwd(s["ids"], case["n"], None, case["n_rows"], s["g"], s["scale"], s["grad"], s["mode"],
                            s["ws"], rows=s["rows"], n_out=s["count"])
            return s["rows"], s["count"], s["grad"]
        if case["mode"] == "add":
            s["grad"].copy_(s["base"])
        sg.sg_embed_bwd(s["ids"], case["n"], None, case["n_rows"], s["g"], s["scale"], s["grad"], s["mode"], s["ws"])
        return s["grad"]
    if op == "xent":
        sg.sg_xent(s["logits"], s["labels"], case["n"], None, s["loss"], s["total"], s["grad"], s["ws"], mean=True)
        return s["loss"], s["total"], s["grad"]
    if op == "orth":
        sg.sg_orthogonalise(s["g"], s["out"], s["ws"], steps=5)
        return s["out"]
    sg.sg_muon_step(s["w"], s["g"], s["m"], s["w_out"], s["m_out"], s["ws"], lr=s["lr"], momentum=s["mu"],
                    nesterov=case["nesterov"], weight_decay=s["wd"], scale=s["scale"], steps=5)
    return s["w_out"], s["m_out"]


def _newton_schulz(u):
    """u: count x rows x cols fp32 -> orthogonalised, five quintic steps."""
    a, b, c = COEF
    x = u / (u.square().sum(dim=(1, 2), keepdim=True).sqrt() + 1e-7)
    tall = x.shape[1] > x.shape[2]
    if tall:
        x = x.transpose(1, 2)
    for _ in range(5):
        p = x @ x.transpose(1, 2)
        x = a * x + (b * p + c * (p @ p)) @ x
    return x.transpose(1, 2) if tall else x


def _run_plain(s):
    case = s["case"]
    op = case["op"]
    if op == "embed_fwd":
        ids = s["ids"].long()
        rows = s["table"][ids.clamp(min=0)].float() * s["scale"]
        return (rows * (ids >= 0)[:, None]).to(DTYPES[case["dtype_out"]])
    if op == "embed_bwd":
        ids, n_rows, dt = s["ids"].long(), case["n_rows"], DTYPES[case["dtype_out"]]
        keep = ids >= 0
        g = s["g"].float() * s["scale"] * keep[:, None]
        if case["mode"] != "rows":
            total = torch.zeros(n_rows, case["dim"], device="cuda")
            total.index_add_(0, ids.clamp(min=0), g)
            return (total + s["base"].float() if case["mode"] == "add" else total).to(dt)
        key, order = torch.sort(torch.where(keep, ids, torch.full_like(ids, n_rows)), stable=True)
        first = torch.ones_like(keep)
        first[1:] = key[1:] != key[:-1]
        first &= key < n_rows
        seg = (torch.cumsum(first, 0) - 1).clamp(min=0)
        grad = torch.zeros(case["n"], case["dim"], device="cuda").index_add_(0, seg, g[order])
        rows = torch.full((case["n"] + 1,), -1, dtype=torch.int32, device="cuda")
        rows[torch.where(first, seg, torch.full_like(seg, case["n"]))] = key.to(torch.int32)
        return rows[:-1], first.sum(dtype=torch.int32).reshape(1), grad.to(dt)
    if op == "xent":
        x, labels = s["logits"].float(), s["labels"].long()
        keep = labels >= 0
        top = x.amax(1, keepdim=True)
        e = torch.exp(x - top)
        z = e.sum(1, keepdim=True)
        at = labels.clamp(min=0)[:, None]
        loss = torch.where(keep, (top + torch.log(z) - x.gather(1, at))[:, 0], torch.zeros_like(z[:, 0]))
        valid = keep.sum().float()
        w = keep.float() / valid.clamp(min=1)
        grad = e / z
        grad.scatter_add_(1, at, torch.full_like(z, -1.0))
        grad *= w[:, None]
        return loss, torch.stack([loss.sum() / valid.clamp(min=1), valid]), grad.to(s["logits"].dtype)
    if op == "orth":
        return _newton_schulz(s["g"].float()).to(s["g"].dtype)
    m = s["mu"] * s["m"] + s["g"]
    u = s["g"] + s["mu"] * m if case["nesterov"] else m
    w = s["w"].float() * (1 - s["lr"] * s["wd"]) - s["lr"] * s["scale"] * _newton_schulz(u)
    return w.to(s["w"].dtype), m


# -------------------------------------------------------------------- exact
def exact(case, seed):
    """The outputs of run() by the operators' definitions in 64 bits."""
    s = _inputs(case, seed)
    op = case["op"]
    if op == "embed_fwd":
        out = torch.zeros(case["n"], case["dim"], dtype=torch.float64, device="cuda")
        at = torch.nonzero(s["ids"] >= 0)[:, 0]
        out[at] = s["table"][s["ids"][at].long()].double() * s["scale"]
        return out
    if op == "embed_bwd":
        at = torch.nonzero(s["ids"] >= 0)[:, 0]
        rows, where = torch.unique(s["ids"][at].long(), sorted=True, return_inverse=True)
        sums = torch.zeros(len(rows), case["dim"], dtype=torch.float64, device="cuda")
        step = max(1, (1 << 28) // case["dim"])  # bounds the 64-bit copies
        for i in range(0, len(at), step):
            sums.index_add_(0, where[i:i + step], s["g"][at[i:i + step]].double())
        sums *= s["scale"]
        if case["mode"] == "rows":
            ids = torch.full((case["n"],), -1, dtype=torch.int32, device="cuda")
            ids[: len(rows)] = rows.to(torch.int32)
            grad = torch.zeros(case["n"], case["dim"], dtype=torch.float64, device="cuda")
            grad[: len(rows)] = sums
            return ids, torch.tensor([len(rows)], dtype=torch.int32, device="cuda"), grad
        if case["mode"] == "add":
            grad = s["base"].double()
        else:
            grad = torch.zeros(case["n_rows"], case["dim"], dtype=torch.float64, device="cuda")
        grad[rows] += sums
        return grad
    if op == "xent":
        x, labels = s["logits"].double(), s["labels"].long()
        logp = x - torch.logsumexp(x, dim=1, keepdim=True)
        good = torch.nonzero(labels >= 0)[:, 0]
        loss = torch.zeros(case["n"], dtype=torch.float64, device="cuda")
        loss[good] = -logp[good, labels[good]]
        n = len(good)
        grad = torch.zeros_like(x)
        if n:
            grad[good] = torch.exp(logp[good]) / n
            grad[good, labels[good]] -= 1.0 / n
        total = torch.stack([loss.sum() / max(1, n), torch.tensor(float(n), dtype=torch.float64, device="cuda")])
        return loss, total, grad
    # an odd polynomial of a matrix acts on its singular values alone: with
    # U = P diag(t) Q^T, f(f(..f(U))) = P diag(f(f(..f(t)))) Q^T
    def polar(u):
        p, t, qt = torch.linalg.svd(u, full_matrices=False)
        t = t / (torch.sqrt(torch.sum(u * u, dim=(1, 2)))[:, None] + 1e-7)
        for _ in range(5):
            t = COEF[0] * t + COEF[1] * t ** 3 + COEF[2] * t ** 5
        return (p * t[:, None, :]) @ qt

    if op == "orth":
        return polar(s["g"].double())
    g = s["g"].double()
    m = s["mu"] * s["m"].double() + g
    o = polar(s["mu"] * m + g if case["nesterov"] else m)
    return s["w"].double() * (1 - s["lr"] * s["wd"]) - s["lr"] * s["scale"] * o, m


# --------------------------------------------------------------------- work
def _distinct(case):
    """Expected number of distinct ids."""
    n, v = 0.99 * case["n"], float(case["n_rows"])
    if not case["skew"]:
        return v * -math.expm1(-n / v)
    total, steps = 0.0, 2000  # integral of 1 - exp(-n p(x)) dx, p(x) = 1 / (x ln(v + 1)), over log x
    h = math.log(v + 1) / steps
    for i in range(steps):
        x = math.exp((i + 0.5) * h)
        total += -math.expm1(-n / (x * math.log(v + 1))) * x * h
    return min(total, n, v)


def work(case):
    op = case["op"]
    size = {"f32": 4, "bf16": 2}
    if op == "embed_fwd":
        n, dim = case["n"], case["dim"]
        return {"bytes": 4 * n + _distinct(case) * dim * size[case["dtype"]] + n * dim * size[case["dtype_out"]],
                "flops": n * dim}
    if op == "embed_bwd":
        n, dim, e = case["n"], case["dim"], size[case["dtype_out"]]
        d = _distinct(case)
        out = {"rows": d * (dim * e + 4), "dense": case["n_rows"] * dim * e,
               "add": 2 * case["n_rows"] * dim * e}[case["mode"]]  # "add" starts from a copy of the given rows
        return {"bytes": 4 * n + n * dim * size[case["dtype"]] + out, "flops": n * dim}
    if op == "xent":
        cells = case["n"] * case["classes"]
        return {"bytes": 2 * cells * size[case["dtype"]] + 8 * case["n"] + 8, "flops": 5 * cells}
    k, m, n = case["count"], min(case["rows"], case["cols"]), max(case["rows"], case["cols"])
    flops = 5 * k * (m * (m + 1) * n + m * m * (m + 1) + 2 * m * m * n)  # the two symmetric products by halves
    e = size[case["dtype"]]
    return {"bytes": k * m * n * (2 * e if op == "orth" else 2 * e + 12), "flops": flops}
