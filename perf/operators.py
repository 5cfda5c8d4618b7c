"""Cases of the training-step operators: the embedding table's lookup and
gradient, matrix products grouped by expert, and distillation from a teacher's
top logits.

`own` chooses what `run` computes with: plain float32 torch operations
(False), or the library's calls (True).  `exact` gives the same outputs from
the definitions in float64.
"""
import math

import numpy as np
import torch

own = False

F32, BF16 = "f32", "bf16"
_DT = {F32: torch.float32, BF16: torch.bfloat16}
_SZ = {F32: 4, BF16: 2}


# ----------------------------------------------------------------- the cases
def listed():
    return [
        # one decoding step of a few sequences: latency alone
        dict(name="lookup_few", kind="lookup", n=4, vocab=32000, dim=768, table=BF16, out=BF16, ids=64),
        # a training batch against a float32 master table, bf16 activations out
        dict(name="lookup_batch", kind="lookup", n=32768, vocab=128000, dim=4096, table=F32, out=BF16, ids=64),
        # a short batch with sides that are no multiples of anything
        dict(name="embed_grad_odd", kind="embed_grad", n=777, vocab=5003, dim=515, dy=F32, dw=F32, ids=32),
        # a training batch's dense float32 table gradient (what AdamW takes)
        dict(name="embed_grad_batch", kind="embed_grad", n=32768, vocab=128000, dim=2048, dy=BF16, dw=F32, ids=64),
        # one decoding step: two experts' rows for each of eight tokens
        dict(name="experts_few_rows", kind="experts", rows=16, experts=16, n=2048, k=1024),
        # a small batch over many experts, some of them empty, ragged row counts
        dict(name="experts_ragged", kind="experts", rows=4133, experts=31, n=1368, k=2056),
        # up projection of the 7B-shaped configuration, eight experts
        dict(name="experts_large", kind="experts", rows=16384, experts=8, n=11008, k=4096),
        # both gradients of a small ragged batch, float32 weight gradients
        dict(name="experts_grad_ragged", kind="experts_grad", rows=4133, experts=24, n=776, k=1032, dw=F32),
        # both gradients of a training batch, 4096 x 4096 experts
        dict(name="experts_grad_large", kind="experts_grad", rows=16384, experts=8, n=4096, k=4096, dw=F32),
        # a few rows: loss and gradient in one call
        dict(name="distill_few", kind="distill", n=8, vocab=32000, top=16, dtype=BF16, temperature=1.0, one_pass=True),
        # a training batch, large vocabulary
        dict(name="distill_batch", kind="distill", n=8192, vocab=128000, top=64, dtype=BF16, temperature=2.0,
             one_pass=True),
        # loss first, gradient later (autograd's order), float32, odd vocabulary
        dict(name="distill_two_calls", kind="distill", n=2047, vocab=50021, top=100, dtype=F32, temperature=1.5,
             one_pass=False),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    """A case of the listed ranges.  Row counts and vocabularies are arbitrary;
    the experts' sides are multiples of 8 (rows on 16-byte boundaries)."""
    kind = rng.choice(["lookup", "embed_grad", "experts", "experts_grad", "distill", "distill"])
    if kind == "lookup":
        return dict(kind=kind, n=_log(rng, 1, 32768), vocab=_log(rng, 1000, 128000), dim=_log(rng, 64, 4096),
                    table=rng.choice([F32, BF16]), out=rng.choice([F32, BF16]), ids=rng.choice([32, 64]))
    if kind == "embed_grad":
        return dict(kind=kind, n=_log(rng, 1, 32768), vocab=_log(rng, 250, 128000), dim=_log(rng, 64, 2048),
                    dy=rng.choice([F32, BF16]), dw=rng.choice([F32, BF16]), ids=rng.choice([32, 64]))
    if kind == "experts":
        return dict(kind=kind, rows=_log(rng, 1, 16384), experts=_log(rng, 1, 64), n=8 * _log(rng, 16, 512),
                    k=8 * _log(rng, 16, 512))
    if kind == "experts_grad":
        return dict(kind=kind, rows=_log(rng, 1, 16384), experts=_log(rng, 1, 32), n=8 * _log(rng, 16, 512),
                    k=8 * _log(rng, 16, 512), dw=rng.choice([F32, BF16]))
    dtype, one_pass, vocab = rng.choice([F32, BF16]), rng.random() < 0.6, _log(rng, 1000, 128000)
    most = (1 << 32) // (vocab * _SZ[dtype] * (2 if one_pass else 3))
    return dict(kind=kind, n=min(_log(rng, 1, 8192), most), vocab=vocab, top=_log(rng, 4, 256), dtype=dtype,
                temperature=rng.choice([0.7, 1.0, 2.0, 4.0]), one_pass=one_pass)


# ------------------------------------------------------------- distributions
_ZIPF_SHIFT = 2.7      # token frequencies go as 1 / (rank + 2.7)


def _zipf_distinct(n, vocab):
    """Expected number of distinct tokens among n."""
    v = np.arange(vocab, dtype=np.float64)
    a = _ZIPF_SHIFT
    p = np.log((v + 1 + a) / (v + a)) / math.log((vocab + a) / a)
    return float(-np.expm1(n * np.log1p(-p)).sum())


def _expert_share(experts):
    """The share of the rows that each expert draws: some are three times as
    popular as others, the last of four or more gets none."""
    p = 1.0 / (1.0 + np.arange(experts) * (2.0 / max(1, experts - 1)))
    if experts >= 4:
        p[-1] = 0.0
    return p / p.sum()


def _expert_used(rows, experts):
    p = _expert_share(experts)
    return float((1.0 - (1.0 - p) ** rows).sum())


def work(case):
    c = case
    if c["kind"] == "lookup":
        used = _zipf_distinct(c["n"], c["vocab"])
        return dict(bytes=used * c["dim"] * _SZ[c["table"]] + c["n"] * (c["dim"] * _SZ[c["out"]] + c["ids"] // 8),
                    flops=c["n"] * c["dim"])
    if c["kind"] == "embed_grad":
        return dict(bytes=c["n"] * (c["dim"] * _SZ[c["dy"]] + c["ids"] // 8) + c["vocab"] * c["dim"] * _SZ[c["dw"]],
                    flops=2 * c["n"] * c["dim"])
    if c["kind"] == "experts":
        used = _expert_used(c["rows"], c["experts"])
        return dict(bytes=2 * (c["rows"] * (c["n"] + c["k"]) + used * c["n"] * c["k"]),
                    flops=2 * c["rows"] * c["n"] * c["k"])
    if c["kind"] == "experts_grad":
        used = _expert_used(c["rows"], c["experts"])
        return dict(bytes=2 * (c["rows"] * (c["n"] + 2 * c["k"]) + used * c["n"] * c["k"])
                    + _SZ[c["dw"]] * c["experts"] * c["n"] * c["k"],
                    flops=4 * c["rows"] * c["n"] * c["k"])
    nv = c["n"] * c["vocab"]
    passes = 2 if c["one_pass"] else 3       # the logits' reads and the gradient's write
    return dict(bytes=passes * nv * _SZ[c["dtype"]] + c["n"] * (c["top"] * (4 + _SZ[c["dtype"]]) + 16),
                flops=(6 if c["one_pass"] else 8) * nv)


# --------------------------------------------------------------- the inputs
def _ids(g, n, vocab, bits):
    """Token ids of natural text: frequency falls with rank; 1 % padding (-1)."""
    a = _ZIPF_SHIFT
    u = torch.rand(n, generator=g, device="cuda", dtype=torch.float64)
    ids = (torch.exp(u * math.log((vocab + a) / a)) * a - a).long().clamp_(0, vocab - 1)
    pad = torch.rand(n, generator=g, device="cuda") < 0.01
    ids[pad] = -1
    return ids if bits == 64 else ids.int()


def _randn(g, shape, dtype, std=1.0):
    x = torch.empty(shape, device="cuda", dtype=torch.float32).normal_(0.0, std, generator=g)
    return x.to(_DT[dtype])


def prepare(case, seed):
    c, g = case, torch.Generator(device="cuda").manual_seed(seed)
    s = dict(c)
    if c["kind"] == "lookup":
        s["ids"] = _ids(g, c["n"], c["vocab"], c["ids"])
        s["W"] = _randn(g, (c["vocab"], c["dim"]), c["table"], 0.02)
        s["Y"] = torch.empty((c["n"], c["dim"]), device="cuda", dtype=_DT[c["out"]])
        s["scale"] = math.sqrt(c["dim"])
    elif c["kind"] == "embed_grad":
        s["ids"] = _ids(g, c["n"], c["vocab"], c["ids"])
        s["dY"] = _randn(g, (c["n"], c["dim"]), c["dy"], 1e-3)
        s["dW"] = torch.empty((c["vocab"], c["dim"]), device="cuda", dtype=_DT[c["dw"]])
        s["scale"] = math.sqrt(c["dim"])
    elif c["kind"] in ("experts", "experts_grad"):
        R, E, N, K = c["rows"], c["experts"], c["n"], c["k"]
        s["sizes"] = np.random.default_rng(seed).multinomial(R, _expert_share(E)).tolist()
        s["offsets"] = torch.tensor(np.concatenate([[0], np.cumsum(s["sizes"])]), device="cuda", dtype=torch.int32)
        s["X"] = _randn(g, (R, K), BF16)
        s["W"] = _randn(g, (E, N, K), BF16, K ** -0.5)
        s["Y"] = torch.empty((R, N), device="cuda", dtype=torch.bfloat16)
        if c["kind"] == "experts_grad":
            s["dY"] = _randn(g, (R, N), BF16, 1e-3)
            s["dX"] = torch.empty((R, K), device="cuda", dtype=torch.bfloat16)
            s["dW"] = torch.empty((E, N, K), device="cuda", dtype=_DT[c["dw"]])
            del s["Y"]
    else:
        n, V, K = c["n"], c["vocab"], c["top"]
        s["logits"] = _randn(g, (n, V), c["dtype"], 2.0)
        # distinct places, the student's logits raised there; one row in eight keeps fewer than K
        first = torch.randint(V, (n, 1), generator=g, device="cuda")
        k = torch.arange(K, device="cuda")
        idx = (first + k * max(1, V // (2 * K)) + (k * k) % max(1, V // (2 * K))) % V
        t = torch.empty((n, K), device="cuda").normal_(0.0, 2.0, generator=g).sort(dim=1, descending=True).values + 6.0
        up = torch.empty((n, K), device="cuda").normal_(0.0, 1.0, generator=g) + t
        s["logits"].scatter_(1, idx, up.to(_DT[c["dtype"]]))
        # a grammar masks one logit in eleven that the teacher does not keep
        if V > 4 * K:
            masked = torch.arange(0, V, 11, device="cuda")
            keep = s["logits"].gather(1, idx)
            s["logits"][:, masked] = float("-inf")
            s["logits"].scatter_(1, idx, keep)
        short = (torch.arange(n, device="cuda") % 8 == 7)[:, None] & (k >= max(1, K // 3))
        s["idx"] = torch.where(short, torch.full_like(idx, -1), idx).int()
        s["teacher"] = t.to(_DT[c["dtype"]])
        w = (torch.rand(n, generator=g, device="cuda") >= 0.05).float()       # prompt rows carry no loss
        s["weight"] = w / n
        s["loss"] = torch.empty(n, device="cuda")
        s["stats"] = torch.empty((n, 2), device="cuda")
        s["dlogits"] = torch.empty_like(s["logits"])
    return s


# ---------------------------------------------------------- the plain forms
def _plain_lookup(s):
    ok = (s["ids"] >= 0) & (s["ids"] < s["vocab"])
    rows = s["W"][torch.where(ok, s["ids"], 0).long()].float() * s["scale"]
    return torch.where(ok[:, None], rows, 0.0).to(s["Y"].dtype)


def _plain_embed_grad(s):
    V = s["vocab"]
    ok = (s["ids"] >= 0) & (s["ids"] < V)
    dW = torch.zeros((V + 1, s["dim"]), device="cuda")                  # the last row takes the padding
    dW.index_add_(0, torch.where(ok, s["ids"], V).long(), s["dY"].float(), alpha=s["scale"])
    return dW[:V].to(s["dW"].dtype)


def _plain_experts(s):
    W = s["W"].float()
    parts = [x.float() @ W[e].T for e, x in enumerate(s["X"].split(s["sizes"]))]
    return torch.cat(parts).to(torch.bfloat16)


def _plain_experts_grad(s):
    W = s["W"].float()
    X, dY = s["X"].float().split(s["sizes"]), s["dY"].float().split(s["sizes"])
    dX = torch.cat([d @ W[e] for e, d in enumerate(dY)]).to(torch.bfloat16)
    dW = torch.stack([d.T @ x for d, x in zip(dY, X)]).to(s["dW"].dtype)
    return dX, dW


def _plain_distill(s):
    T, V = s["temperature"], s["vocab"]
    w = s["weight"][:, None]
    present = (s["idx"] >= 0) & (s["idx"] < V)
    idx = torch.where(present, s["idx"], 0).long()
    t = torch.where(present, s["teacher"].float(), float("-inf"))
    t = (t - t.amax(1, keepdim=True)) / T
    e = torch.exp(t)
    z = e.sum(1, keepdim=True)
    p, logp = e / z, t - torch.log(z)
    x = s["logits"].float()
    x = (x - x.amax(1, keepdim=True)) / T
    ex = torch.exp(x)
    zx = ex.sum(1, keepdim=True)
    logq = x.gather(1, idx) - torch.log(zx)
    terms = torch.where(p > 0, p * (logp - logq), 0.0)
    loss = torch.where(w[:, 0] != 0, T * T * w[:, 0] * terms.sum(1), 0.0)
    grad = ex / zx
    grad.scatter_add_(1, idx, -p)
    grad = torch.where(w != 0, (T * w) * grad, 0.0)
    return loss, grad.to(s["logits"].dtype)


# ------------------------------------------------------------------ one pass
def _workspace(s, nbytes, *sizes):
    """The call's workspace, kept with the state as a program keeps it."""
    if "ws" not in s:
        s["ws"] = torch.zeros(nbytes(*sizes), device="cuda", dtype=torch.uint8)
    return s["ws"]


def run(state):
    s = state
    if not own:
        return {"lookup": _plain_lookup, "embed_grad": _plain_embed_grad, "experts": _plain_experts,
                "experts_grad": _plain_experts_grad, "distill": _plain_distill}[s["kind"]](s)
    import matrix_optimizers_gb300 as mo
    if s["kind"] == "lookup":
        mo.embedding_lookup(s["W"], s["ids"], s["Y"], scale=s["scale"])
        return s["Y"]
    if s["kind"] == "embed_grad":
        ws = _workspace(s, mo.embedding_grad_workspace_bytes, s["n"], s["vocab"], s["dim"])
        mo.embedding_grad(s["dY"], s["ids"], s["dW"], ws, scale=s["scale"])
        return s["dW"]
    if s["kind"] in ("experts", "experts_grad"):
        ws = _workspace(s, mo.expert_linear_workspace_bytes, s["rows"], s["n"], s["k"], s["experts"])
        if s["kind"] == "experts":
            mo.expert_linear(s["X"], s["W"], s["offsets"], s["Y"], ws)
            return s["Y"]
        mo.expert_linear_dgrad(s["dY"], s["W"], s["offsets"], s["dX"], ws)
        mo.expert_linear_wgrad(s["dY"], s["X"], s["offsets"], s["dW"], ws)
        return s["dX"], s["dW"]
    if s["one_pass"]:
        mo.distill_topk_loss_grad(s["logits"], s["idx"], s["teacher"], s["loss"], s["dlogits"],
                                  temperature=s["temperature"], row_weight=s["weight"])
    else:
        mo.distill_topk_loss(s["logits"], s["idx"], s["teacher"], s["loss"], s["stats"],
                             temperature=s["temperature"], row_weight=s["weight"])
        mo.distill_topk_grad(s["logits"], s["idx"], s["teacher"], s["stats"], s["dlogits"],
                             temperature=s["temperature"], row_weight=s["weight"])
    return s["loss"], s["dlogits"]


# ------------------------------------------------- the definitions in 64 bits
def _exact_embed_grad(s):
    """Sorted by token, a token's rows are the difference of two running sums."""
    V = s["vocab"]
    ids = s["ids"].long()
    ids = torch.where((ids < 0) | (ids >= V), V, ids)
    key, order = torch.sort(ids)
    ends = torch.searchsorted(key, torch.arange(V + 1, device="cuda"))
    run_ = torch.zeros((len(ids) + 1, s["dim"]), device="cuda", dtype=torch.float64)
    torch.cumsum(s["dY"][order].double(), 0, out=run_[1:])
    return (run_[ends[1:]] - run_[ends[:-1]]) * s["scale"]


def _exact_distill(s):
    T, V, n = s["temperature"], s["vocab"], s["n"]
    loss = torch.zeros(n, device="cuda", dtype=torch.float64)
    grad = torch.zeros((n, V), device="cuda", dtype=torch.float64)
    step = max(1, (1 << 27) // V)
    for a in range(0, n, step):
        rows = slice(a, min(n, a + step))
        w = s["weight"][rows].double()[:, None]
        idx = s["idx"][rows].long()
        absent = (idx < 0) | (idx >= V)
        t = (s["teacher"][rows].double() / T).masked_fill(absent, float("-inf"))
        logp = torch.log_softmax(t, 1)
        logq = torch.log_softmax(s["logits"][rows].double() / T, 1)
        p = logp.exp()
        at = idx.masked_fill(absent, 0)
        kl = torch.where(absent, 0.0, p * (logp - logq.gather(1, at))).sum(1)
        loss[rows] = T * T * w[:, 0] * kl
        grad[rows] = T * w * logq.exp().scatter_add(1, at, -p)
    return loss, grad


def exact(case, seed):
    s = prepare(case, seed)
    if s["kind"] == "lookup":
        W = torch.cat([s["W"].double(), torch.zeros((1, s["dim"]), device="cuda", dtype=torch.float64)])
        return W[s["ids"].long()] * s["scale"]                          # padding (-1) takes the last row
    if s["kind"] == "embed_grad":
        return _exact_embed_grad(s)
    if s["kind"] == "distill":
        return _exact_distill(s)
    of = torch.repeat_interleave(torch.arange(s["experts"], device="cuda"),
                                 torch.tensor(s["sizes"], device="cuda"))
    if s["kind"] == "experts":
        Y = torch.zeros((s["rows"], s["n"]), device="cuda", dtype=torch.float64)
        for e in range(s["experts"]):
            at = (of == e).nonzero()[:, 0]
            Y[at] = torch.mm(s["X"][at].double(), s["W"][e].double().t())
        return Y
    dX = torch.zeros((s["rows"], s["k"]), device="cuda", dtype=torch.float64)
    dW = torch.zeros((s["experts"], s["n"], s["k"]), device="cuda", dtype=torch.float64)
    for e in range(s["experts"]):
        at = (of == e).nonzero()[:, 0]
        dX[at] = torch.mm(s["dY"][at].double(), s["W"][e].double())
        dW[e] = torch.mm(s["dY"][at].double().t(), s["X"][at].double())
    return dX, dW
