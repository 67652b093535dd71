"""Operators around the classifier's logits and the layers' states, as cases
with their inputs, their plain form in torch and the calls a user of the
package makes.

A case is a dict of plain values; "op" names the operator:
  logprobs  per row of logits: the log probability of a given class, the
            entropy, and the k most probable classes with their log
            probabilities (ties to the lowest class; classes at -inf take no
            part: entries past the others hold class -1 and -inf)
  distill   distillation from a teacher's top logits: per row
            T^2 KL(q || p), q the softmax of the teacher's k values / T, p that
            of the student's logits / T over all classes; its mean over the
            rows with a teacher, and the gradient
  ln_fwd    layer norm of rows, with the rows' mean and 1 / deviation
  ln_bwd    its gradient: of the rows, the weight and the bias
"""
import math

import torch

own = False

DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16}
SIZE = {"f32": 4, "bf16": 2}
EPS = 1e-5


def listed():
    return [
        # the answers of one batch of seeds: as many classes as the hidden width
        dict(name="logprobs_seeds", op="logprobs", n=256, classes=128, k=5, dtype="f32", masked="none"),
        # the answers of a whole graph's nodes, a chunk at a time, over an odd number of classes
        dict(name="logprobs_nodes", op="logprobs", n=200001, classes=47, k=3, dtype="f32", masked="none"),
        # serving: a few rows over a very long axis, some classes not to be answered with
        dict(name="logprobs_long", op="logprobs", n=4, classes=131072, k=20, dtype="f32", masked="inf"),
        # a teacher's pass: the top logits of many rows over an odd number of classes
        dict(name="logprobs_teacher", op="logprobs", n=4096, classes=50257, k=64, dtype="bf16", masked="none"),
        # one batch of seeds learning from a teacher
        dict(name="distill_seeds", op="distill", n=256, classes=128, k=8, dtype="f32", temperature=2.0, masked="none"),
        # a few rows over a very long axis, classes masked by the type's lowest value
        dict(name="distill_long", op="distill", n=5, classes=131072, k=64, dtype="f32", temperature=1.0, masked="low"),
        # a large batch over an odd number of classes (rows start at any 2-byte address)
        dict(name="distill_large", op="distill", n=4096, classes=50257, k=64, dtype="bf16", temperature=2.0,
             masked="none"),
        # the hidden states of one batch of seeds
        dict(name="ln_fwd_seeds", op="ln_fwd", n=256, dim=128, dtype="f32", dtype_w="f32"),
        # states of an odd width: rows start at any 2-byte address
        dict(name="ln_fwd_odd", op="ln_fwd", n=30011, dim=1001, dtype="bf16", dtype_w="f32"),
        # the gradient of a small batch's states
        dict(name="ln_bwd_seeds", op="ln_bwd", n=1024, dim=128, dtype="f32", dtype_w="f32"),
        # the gradient of the states of a three-hop batch's nodes
        dict(name="ln_bwd_batch", op="ln_bwd", n=600001, dim=128, dtype="f32", dtype_w="f32"),
        # wide states in bf16, weights as well
        dict(name="ln_bwd_wide", op="ln_bwd", n=16384, dim=4096, dtype="bf16", dtype_w="bf16"),
    ]


def _log_int(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["logprobs", "logprobs", "distill", "distill", "ln_fwd", "ln_bwd"])
    dtype = rng.choice(["f32", "bf16"])
    if op in ("logprobs", "distill"):
        classes = rng.choice([_log_int(rng, 2, 200000), _log_int(rng, 2, 200000), 128, 50257])
        n = _log_int(rng, 1, min(200000, (200000000 if dtype == "bf16" else 100000000) // classes))
        case = dict(op=op, n=n, classes=classes, k=_log_int(rng, 1, min(128, classes)), dtype=dtype,
                    masked=rng.choice(["none", "none", "inf", "low"]))
        if op == "distill":
            case["temperature"] = rng.choice([1.0, 2.0, 4.0])
        return case
    dim = rng.choice([_log_int(rng, 1, 16384), _log_int(rng, 1, 16384), 64, 100, 128, 256, 1024])
    most = min(600000, (128000000 if dtype == "bf16" else 64000000) // dim)
    return dict(op=op, n=_log_int(rng, 1, most), dim=dim, dtype=dtype, dtype_w=rng.choice(["f32", dtype]))


# ------------------------------------------------------------------- inputs
def _generator(seed, salt):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed * 1000003 + salt)
    return g


def _masked(case, x, keep, g):
    """x with a tenth of the classes that `keep` does not name masked; with
    -inf, one row in a hundred has nothing left."""
    if case["masked"] == "none":
        return x
    off = torch.rand(x.shape, generator=g, device="cuda") < 0.1
    if keep is not None:
        off.scatter_(1, keep, False)
    if case["masked"] == "low":
        return x.masked_fill_(off, torch.finfo(DTYPES[case["dtype"]]).min)
    if keep is None:
        off |= (torch.rand(len(x), generator=g, device="cuda") < 0.01)[:, None]
    return x.masked_fill_(off, float("-inf"))


def _inputs(case, seed):
    op, n, dt = case["op"], case["n"], DTYPES[case["dtype"]]
    if op == "logprobs":
        g = _generator(seed, 1)
        c = case["classes"]
        x = torch.empty(n, c, device="cuda").normal_(0, 2, generator=g)
        labels = torch.randint(0, c, (n,), generator=g, device="cuda", dtype=torch.int32)
        x.scatter_add_(1, labels.long()[:, None], torch.full((n, 1), 3.0, device="cuda"))
        x = _masked(case, x, None, g).to(dt)
        none = torch.rand(n, generator=g, device="cuda") < 0.02
        return dict(logits=x, labels=labels.masked_fill_(none, -1))
    if op == "distill":
        g = _generator(seed, 2)
        c, k = case["classes"], case["k"]
        # k distinct classes of each row, their values in descending order;
        # one row in ten has fewer, one in fifty none
        start = torch.randint(0, c, (n, 1), generator=g, device="cuda")
        ids = (start + torch.arange(k, device="cuda") * (c // k)) % c
        values = torch.sort(torch.empty(n, k, device="cuda").normal_(5, 3, generator=g), dim=1, descending=True)[0]
        x = torch.empty(n, c, device="cuda").normal_(0, 2, generator=g)
        x.scatter_add_(1, ids, 0.7 * values)
        x = _masked(case, x, ids, g).to(dt)
        u = torch.rand(n, 2, generator=g, device="cuda")
        left = torch.where(u[:, 0] < 0.1, (u[:, 1] * k).long() + 1, torch.full((n,), k, device="cuda"))
        left = left.masked_fill(u[:, 0] > 0.98, 0).clamp(max=k)
        ids = torch.where(torch.arange(k, device="cuda") < left[:, None], ids, torch.full_like(ids, -1))
        return dict(logits=x, ids=ids.to(torch.int32), values=values)
    g = _generator(seed, 3 if op == "ln_fwd" else 4)
    d, dw = case["dim"], DTYPES[case["dtype_w"]]
    x = torch.empty(n, d, device="cuda").normal_(generator=g)
    x *= 0.5 + torch.rand(n, 1, generator=g, device="cuda")
    x += torch.empty(n, 1, device="cuda").normal_(generator=g)
    out = dict(x=x.to(dt), weight=(1 + 0.1 * torch.randn(d, generator=g, device="cuda")).to(dw))
    if op == "ln_fwd":
        out["bias"] = (0.1 * torch.randn(d, generator=g, device="cuda")).to(dw)
        return out
    x = out["x"].float()
    out["mean"] = x.mean(1)
    out["rstd"] = torch.rsqrt((x - out["mean"][:, None]).square().mean(1) + EPS)
    out["g"] = (1e-3 * torch.empty(n, d, device="cuda").normal_(generator=g)).to(dt)
    return out


def prepare(case, seed):
    state = dict(case=case, **_inputs(case, seed))
    if not own:
        return state
    # the outputs and workspaces that a program keeps from step to step
    from sampling_gnn_mini_gb300 import binding as sg
    op, n = case["op"], case["n"]
    state["sg"] = sg

    def f32(*shape):
        return torch.empty(shape, device="cuda")
    if op == "logprobs":
        state.update(logp=f32(n), entropy=f32(n), top_logp=f32(n, case["k"]),
                     top_ids=torch.empty(n, case["k"], dtype=torch.int32, device="cuda"))
    elif op == "distill":
        state.update(loss=f32(n), total=f32(2), grad=torch.empty_like(state["logits"]),
                     ws=sg.aligned_workspace(sg.sg_distill_workspace(n, case["classes"])))
    elif op == "ln_fwd":
        state.update(out=torch.empty_like(state["x"]), mean=f32(n), rstd=f32(n))
    else:
        state.update(dx=torch.empty_like(state["x"]), dweight=torch.empty_like(state["weight"]),
                     dbias=torch.empty_like(state["weight"]),
                     ws=sg.aligned_workspace(sg.sg_layernorm_bwd_workspace(n, case["dim"])))
    return state


# --------------------------------------------------------------------- run
def run(state):
    return _run_own(state) if own else _run_plain(state)


def _run_own(s):
    sg, case = s["sg"], s["case"]
    op, n = case["op"], case["n"]
    if op == "logprobs":
        sg.sg_logprobs(s["logits"], s["labels"], n, None, s["logp"], s["entropy"], s["top_ids"], s["top_logp"])
        return s["logp"], s["entropy"], s["top_ids"], s["top_logp"]
    if op == "distill":
        sg.sg_distill(s["logits"], s["ids"], s["values"], n, None, s["loss"], s["total"], s["grad"], s["ws"],
                      temperature=case["temperature"], mean=True)
        return s["loss"], s["total"], s["grad"]
    if op == "ln_fwd":
        sg.sg_layernorm_fwd(s["x"], s["weight"], s["bias"], n, None, s["out"], mean=s["mean"], rstd=s["rstd"], eps=EPS)
        return s["out"], s["mean"], s["rstd"]
    sg.sg_layernorm_bwd(s["g"], s["x"], s["weight"], s["mean"], s["rstd"], n, None, s["dx"], s["dweight"], s["dbias"],
                        s["ws"])
    return s["dx"], s["dweight"], s["dbias"]


def _exp(x):
    """max of each row (0 where nothing is left), max - x, exp(x - max) and its sum."""
    m = x.amax(1, keepdim=True)
    m = torch.where(m == float("-inf"), torch.zeros_like(m), m)
    d = m - x
    e = torch.exp(-d)
    return m, d, e, e.sum(1, keepdim=True)


def _top(x, k):
    """The k largest of each row with their classes: unique 64-bit keys, the
    value's bits in an order that whole numbers share, then the class."""
    bits = (x + 0.0).view(torch.int32)
    order = torch.where(bits < 0, bits ^ 0x7FFFFFFF, bits).long()
    key = (order << 32) | (0x7FFFFFFF - torch.arange(x.shape[1], device=x.device))
    ids = 0x7FFFFFFF - (torch.topk(key, k, dim=1)[0] & 0x7FFFFFFF)
    return ids, x.gather(1, ids)


def _run_plain(s):
    case = s["case"]
    op = case["op"]
    if op == "logprobs":
        x, labels = s["logits"].float(), s["labels"].long()
        m, d, e, z = _exp(x)
        log_z = torch.log(z)
        logp = (x.gather(1, labels.clamp(min=0)[:, None]) - m - log_z)[:, 0]
        logp = torch.where(labels < 0, torch.zeros_like(logp), torch.where(z[:, 0] == 0, float("-inf"), logp))
        entropy = (log_z + torch.where(e > 0, e * d, torch.zeros_like(e)).sum(1, keepdim=True) / z)[:, 0]
        entropy = torch.where(z[:, 0] == 0, torch.zeros_like(entropy), entropy)
        ids, top = _top(x, case["k"])
        gone = top == float("-inf")
        top = torch.where(gone, top, top - m - log_z)
        return logp, entropy, torch.where(gone, -1, ids).to(torch.int32), top
    if op == "distill":
        t, ids, k = case["temperature"], s["ids"].long(), case["k"]
        used = ids[:, :1] >= 0
        v = torch.where(ids >= 0, s["values"], float("-inf"))
        vm, vd, ve, vz = _exp(v / t)
        q = torch.where(used, ve / vz, torch.zeros_like(ve))
        log_q = torch.where(q > 0, -vd - torch.log(vz), torch.zeros_like(vd))
        x = s["logits"].float() / t
        m, d, e, z = _exp(x)
        at = ids.clamp(min=0)
        log_p = torch.where(q > 0, x.gather(1, at) - m - torch.log(z), torch.zeros_like(q))
        loss = t * t * (q * (log_q - log_p)).sum(1)
        rows = used.sum().float()
        w = used / rows.clamp(min=1)
        grad = (e / z).scatter_add_(1, at, -q) * (t * w)
        return loss, torch.stack([loss.sum() / rows.clamp(min=1), rows]), grad.to(s["logits"].dtype)
    x, w = s["x"].float(), s["weight"].float()
    if op == "ln_fwd":
        mean = x.mean(1)
        h = x - mean[:, None]
        rstd = torch.rsqrt(h.square().mean(1) + EPS)
        return (h * rstd[:, None] * w + s["bias"].float()).to(s["x"].dtype), mean, rstd
    g, rstd = s["g"].float(), s["rstd"][:, None]
    h = (x - s["mean"][:, None]) * rstd
    gw = g * w
    dx = rstd * (gw - gw.mean(1, keepdim=True) - h * (gw * h).mean(1, keepdim=True))
    return dx.to(s["x"].dtype), (g * h).sum(0).to(s["weight"].dtype), g.sum(0).to(s["weight"].dtype)


# -------------------------------------------------------------------- exact
def exact(case, seed):
    """The outputs of run() by the operators' definitions in 64 bits."""
    s = _inputs(case, seed)
    op, n = case["op"], case["n"]
    inf = float("inf")
    if op == "logprobs":
        x = s["logits"].double()
        lse = torch.logsumexp(x, dim=1)
        logp_all = x - torch.where(lse == -inf, torch.zeros_like(lse), lse)[:, None]
        at = s["labels"].long()
        logp = torch.where(at >= 0, logp_all[torch.arange(n, device="cuda"), at.clamp(min=0)], 0.0)
        entropy = torch.special.entr(torch.exp(logp_all)).sum(1)
        top = torch.sort(torch.topk(logp_all, case["k"], dim=1)[0], dim=1, descending=True)[0]
        return logp, entropy, None, top
    if op == "distill":
        t = case["temperature"]
        there = (s["ids"] >= 0) & (s["ids"][:, :1] >= 0)
        q = torch.zeros(n, case["classes"], dtype=torch.float64, device="cuda")
        row, col = torch.nonzero(there, as_tuple=True)
        share = torch.exp(torch.log_softmax(torch.where(there, s["values"].double(), -inf) / t, dim=1))
        q[row, s["ids"][row, col].long()] = share[row, col]
        logp = torch.log_softmax(s["logits"].double() / t, dim=1)
        loss = t * t * torch.where(q > 0, q * (torch.log(q) - logp), 0.0).sum(1)
        used = s["ids"][:, 0] >= 0
        count = max(1, int(used.sum()))
        grad = torch.exp(logp).sub_(q).mul_((used * (t / count))[:, None])
        total = torch.stack([loss.sum() / count, used.sum().double()])
        return loss, total, grad
    x, w = s["x"].double(), s["weight"].double()
    if op == "ln_fwd":
        var, mean = torch.var_mean(x, dim=1, correction=0)
        rstd = 1 / torch.sqrt(var + EPS)
        return torch.addcmul(s["bias"].double(), (x - mean[:, None]) * rstd[:, None], w), mean, rstd
    g, r = s["g"].double(), s["rstd"].double()[:, None]
    h = (x - s["mean"].double()[:, None]) * r
    # the Jacobian of a row, r (I - 1 1^T / d - h h^T / d), on g w
    a = g * w
    dot = torch.einsum("nd,nd->n", a, h)[:, None]
    dx = r * (a - (a.sum(1, keepdim=True) + h * dot) / case["dim"])
    return dx, torch.einsum("nd,nd->d", g, h), g.sum(0)


# --------------------------------------------------------------------- work
def work(case):
    n, e = case["n"], SIZE[case["dtype"]]
    if case["op"] in ("logprobs", "distill"):
        cells, k = n * case["classes"], case["k"]
        if case["op"] == "logprobs":
            return {"bytes": cells * e + 12 * n + 8 * n * k, "flops": 6 * cells}
        return {"bytes": 2 * cells * e + 8 * n * k + 4 * n + 8, "flops": 5 * cells}
    cells, d, ew = n * case["dim"], case["dim"], SIZE[case["dtype_w"]]
    if case["op"] == "ln_fwd":
        return {"bytes": 2 * cells * e + 8 * n + 2 * d * ew, "flops": 8 * cells}
    return {"bytes": 3 * cells * e + 8 * n + 3 * d * ew, "flops": 14 * cells}
