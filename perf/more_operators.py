"""The two ends of a distillation step of a whole model, as cases that can be timed and checked.

Log probabilities of given tokens with the entropy and the most likely tokens
(what a teacher's pass hands to the distillation loss, and what scores an
answer), from logits and from hidden states, with their gradients; and the
norm of all gradients of a model with the clipping by it.  ``run`` computes
them in plain torch operations in 32 bits (long sums of squares in 64), or,
with ``own``, through the library's entry points; ``exact`` gives the same
values from the definitions in 64 bits.

Sizes are the repository's own (hidden 2048, vocabulary 151936, the teacher's
top 64, 16384 tokens, the scales of a layer of 128 experts of 2048 x 768) and
generic ones.

Ids are compared as whole numbers, so which logit is larger must not hang on
the order of a sum: hidden states and output weights lie on the grid of an INT8
quantiser whose scale is a power of two (clamped normal values, 32 steps of
standard deviation).  Every partial sum of such products is a whole number of
steps below 2^24, exact in 32 bits in any order; ties occur and go to the
lowest id.
"""
import math
import random

import torch

own = False

BF = torch.bfloat16
F32 = torch.float32
STEPS = 32.0                       # standard deviation of the integer grids


# ------------------------------------------------------------------- cases --
def listed():
    return [
        # one served token: its log probability, entropy and 20 alternatives from a row of logits (latency)
        dict(name="logits_token", op="logits", T=1, V=151936, m=1, k=20, ent=True, masked=False),
        # a sequence of the distillation's logits: the teacher's top 64, labels' log probabilities
        dict(name="logits_sequence", op="logits", T=2048, V=151936, m=1, k=64, ent=False, masked=False),
        # the gradient of log probabilities and entropies on a ragged batch of logits, odd vocabulary
        dict(name="logits_grad", op="logits_grad", T=777, V=50257, m=1, ent=True, masked=False),
        # one served token from its hidden state: the whole output weight for one row
        dict(name="head_token", op="head", T=1, H=2048, V=151936, m=1, k=20, ent=True),
        # a short answer scored under a mid-sized vocabulary, odd sizes
        dict(name="head_short", op="head", T=333, H=1024, V=32003, m=1, k=5, ent=True),
        # the teacher's pass over one sequence of a distillation step
        dict(name="head_sequence", op="head", T=2048, H=2048, V=151936, m=0, k=64, ent=False),
        # the teacher's pass over the whole batch, with the labels scored on the way
        dict(name="head_batch", op="head", T=16384, H=2048, V=151936, m=1, k=64, ent=True),
        # a sequence trained on weighted log probabilities with an entropy term
        dict(name="head_grad", op="head_grad", T=2048, H=2048, V=151936, m=1, ent=True),
        # the same on a short answer, log probabilities alone
        dict(name="head_grad_short", op="head_grad", T=333, H=1024, V=32003, m=1, ent=False),
        # 64 gradients of 128 activation scales each: launches and latency
        dict(name="clip_scales", op="clip", kind="even", n=64, size=128, dtype="fp32", shapes=0),
        # a ragged list of bf16 gradients (odd lengths, odd addresses)
        dict(name="clip_ragged", op="clip", kind="ragged", n=311, size=60000, dtype="bf16", shapes=7),
        # the scale gradients of eight expert layers, four tensors each
        dict(name="clip_model", op="clip", kind="layers", n=32, size=0, dtype="fp32", shapes=0),
    ]


def _log(rng, lo, hi, step=1):
    v = math.exp(rng.uniform(math.log(lo), math.log(hi + 0.999)))
    return max(step, int(v) // step * step)


def draw(rng):
    op = rng.choice(["logits", "logits", "logits_grad", "head", "head", "head_grad", "clip"])
    V = _log(rng, 1000, 151936)
    m = rng.choice([0, 1, 1, 3])
    ent = rng.random() < 0.6
    if op == "logits":
        return dict(op=op, T=_log(rng, 1, 2048), V=V, m=m, k=rng.choice([0, 1, 5, 20, 33, 64]), ent=ent or m == 0,
                    masked=rng.random() < 0.3)
    if op == "logits_grad":
        return dict(op=op, T=_log(rng, 1, 2048), V=V, m=max(m, 1), ent=ent, masked=rng.random() < 0.3)
    if op == "head":
        return dict(op=op, T=_log(rng, 1, 4096), H=_log(rng, 128, 4096, 64), V=V, m=m,
                    k=rng.choice([0, 1, 5, 20, 33, 64]), ent=ent or m == 0)
    if op == "head_grad":
        return dict(op=op, T=_log(rng, 1, 4096), H=_log(rng, 128, 4096, 64), V=V, m=max(m, 1), ent=ent)
    n = _log(rng, 1, 600)
    return dict(op=op, kind="ragged", n=n, size=_log(rng, 1, min(4_000_000, 100_000_000 // n)),
                dtype=rng.choice(["fp32", "bf16", "mixed"]), shapes=rng.randrange(1, 1 << 20))


def _lengths(case):
    """The tensors of a clip case: (length, bf16 or not, offset of the first element in its buffer)."""
    n, size = case["n"], case["size"]
    if case["kind"] == "layers":                                     # ds_w1, ds_w2 (one per 16), ds_a1, ds_a2
        return [(s, False, 0) for s in (128 * 1536 * 128, 128 * 2048 * 48, 128, 128)] * (n // 4)
    if case["kind"] == "even":
        return [(size, case["dtype"] == "bf16", 0)] * n
    rng = random.Random(case["shapes"])
    out = []
    for _ in range(n):
        bf = case["dtype"] == "bf16" or (case["dtype"] == "mixed" and rng.random() < 0.5)
        out.append((_log(rng, max(1, size // 30), size), bf, rng.choice([0, 0, 0, 1, 3])))
    return out


def work(case):
    c, op = case, case["op"]
    if op == "clip":
        t = _lengths(c)
        return dict(bytes=sum((6 if bf else 12) * n for n, bf, _ in t), flops=3 * sum(n for n, _, _ in t))
    T, V, m = c["T"], c["V"], c["m"]
    small = T * (4 + 4 * c["ent"] + 8 * m + 8 * c.get("k", 0))
    if op == "logits":
        return dict(bytes=2 * T * V + small, flops=6 * T * V)
    if op == "logits_grad":
        return dict(bytes=4 * T * V + small, flops=6 * T * V)
    H = c["H"]
    if op == "head":
        return dict(bytes=2 * V * H + 2 * T * H + small, flops=2 * T * V * H)
    return dict(bytes=2 * V * H + 4 * T * H + small, flops=4 * T * V * H)


# ------------------------------------------------------------------ inputs --
def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _randn(g, *shape):
    return torch.randn(shape, generator=g, device="cuda")


def _rand_ids(g, V, *shape):
    return torch.randint(0, V, shape, generator=g, device="cuda")


def _padded(g, ids):
    """The first given token of a row in twenty is padding (-1), but never the only row's."""
    if ids.shape[0] > 1 and ids.shape[1]:
        ids[torch.rand((ids.shape[0],), generator=g, device="cuda") < 0.05, 0] = -1
    return ids.to(torch.int32)


def prepare(case, seed):
    g, c, op = _gen(seed), case, case["op"]
    s = dict(case=c)
    if op == "clip":
        s["grads"] = []
        for n, bf, off in _lengths(c):
            buf = _randn(g, n + off) * math.exp(2.0 * math.sin(1.7 * len(s["grads"])) - 5.0)
            s["grads"].append(buf.to(BF if bf else F32)[off:])
        total = sum(n for n, _, _ in _lengths(c))
        s["max_norm"] = 0.002 * math.sqrt(total)                     # below the norm: the step is clipped
        return s
    T, V, m = c["T"], c["V"], c["m"]
    if op.startswith("logits"):
        ids = _rand_ids(g, V, T, m)
        ld = (V + 7) // 8 * 8                                        # rows padded to whole vectors
        sure = torch.rand((T, 1), generator=g, device="cuda") * 12.0
        z = torch.empty((T, ld), dtype=BF, device="cuda")
        for r in range(0, T, 1024):
            part = _randn(g, min(1024, T - r), ld) * 2.0
            if c["masked"]:                                          # tokens a grammar rules out
                part.masked_fill_(torch.rand(part.shape, generator=g, device="cuda") < 0.3, -math.inf)
            if m:
                part.scatter_(1, ids[r:r + 1024], _randn(g, part.shape[0], m) + sure[r:r + 1024])
            z[r:r + 1024] = part.to(BF)
        s["z"] = z[:, :V]
    else:
        H = c["H"]
        unit = 2.0 ** round(math.log2(2.0 / (STEPS * STEPS * math.sqrt(H))))   # of a logit: deviation about 2
        wq = torch.round(_randn(g, V, H) * STEPS).clamp_(-127, 127)
        ids = _rand_ids(g, V, T, m)
        hq = _randn(g, T, H) * STEPS
        if m:                                                        # how much the first given token stands out
            hq += torch.rand((T, 1), generator=g, device="cuda") * (12.0 / (unit * STEPS * STEPS * H)) * wq[ids[:, 0]]
        s["w"] = (wq * (unit * 32)).to(BF)
        s["h"] = (torch.round(hq).clamp_(-127, 127) / 32).to(BF)
        del wq, hq
    s["ids"] = _padded(g, ids) if m else None
    if op.endswith("grad"):
        # a program's upstream gradients: advantages over the tokens, a weight on the entropy
        s["dlogp"] = _randn(g, T, m) / T
        s["dent"] = (0.1 + 0.02 * _randn(g, T)) / T if c["ent"] else None
        # what the forward pass left
        lse, ent = torch.empty(T, device="cuda"), torch.empty(T, device="cuda")
        for r in range(0, T, 512):
            z = _logits(s, slice(r, r + 512), F32).double()
            lse[r:r + 512] = torch.logsumexp(z, -1).float()
            p = torch.softmax(z, -1)
            ent[r:r + 512] = -torch.where(p > 0, p * torch.log(p), p).sum(-1).float()
        s["lse"], s["entropy"] = lse, ent if c["ent"] else None
    return s


# -------------------------------------------------------------- plain forms --
def _logits(st, rows, ft):
    if "z" in st:
        return st["z"][rows].to(ft)
    return st["h"][rows].to(ft) @ st["w"].to(ft).t()


def _parts(st):
    """Row ranges whose logits in 32 bits take about 4 GB."""
    T, V = st["case"]["T"], st["case"]["V"]
    n = max(1, (1 << 30) // V)
    return [slice(r, min(r + n, T)) for r in range(0, T, n)]


def _ranked(z):
    """One whole number per logit, larger for a larger logit and, among equals, for the lower id."""
    b = (z + 0.0).view(torch.int32)                                  # -0 counts as 0
    b = torch.where(b < 0, b ^ 0x7fffffff, b).long()
    return (b << 32) + (0x7fffffff - torch.arange(z.shape[1], device=z.device))


def _forward(st):
    c, ids = st["case"], st["ids"]
    k, V = c["k"], c["V"]
    out = dict(lse=[], entropy=[], logp=[], top_ids=[], top_logp=[])
    for rows in _parts(st):
        z = _logits(st, rows, F32)
        m = z.amax(-1, keepdim=True)
        e = torch.exp(z - m)
        S = e.sum(-1, keepdim=True)
        lse = m + torch.log(S)
        out["lse"].append(lse[:, 0])
        if c["ent"]:
            out["entropy"].append((torch.log(S) - torch.where(e > 0, e * (z - m), 0.0).sum(-1, keepdim=True) / S)[:, 0])
        del e
        if c["m"]:
            i = ids[rows].long()
            ok = (i >= 0) & (i < V)
            out["logp"].append(torch.where(ok, z.gather(1, i.clamp(0, V - 1)) - lse, 0.0))
        if k:
            top = 0x7fffffff - (torch.topk(_ranked(z), k, -1).values & 0xffffffff)
            v = z.gather(1, top)
            out["top_ids"].append(torch.where(v > -math.inf, top, -1).to(torch.int32))
            out["top_logp"].append(v - lse)
    return {n: torch.cat(v) if v else None for n, v in out.items()}


def _backward(st):
    c, ids = st["case"], st["ids"]
    T, V = c["T"], c["V"]
    grad = torch.empty((T, c.get("H", V)), dtype=BF, device="cuda")
    for rows in _parts(st):
        z = _logits(st, rows, F32)
        i = ids[rows].long()
        ok = (i >= 0) & (i < V)
        a = torch.where(ok, st["dlogp"][rows], 0.0)
        lp = z - st["lse"][rows, None]
        f = a.sum(-1, keepdim=True)
        if c["ent"]:
            f = f + st["dent"][rows, None] * (torch.where(lp > -math.inf, lp, 0.0) + st["entropy"][rows, None])
        d = (-torch.exp(lp) * f).scatter_add_(1, i.clamp(0, V - 1), a)
        grad[rows] = (d if "z" in st else d @ st["w"].float()).to(BF)
    return grad


def _clip(st):
    total = torch.zeros((), dtype=torch.float64, device="cuda")
    for g in st["grads"]:
        total = total + g.double().square().sum()
    norm = torch.sqrt(total)
    f = torch.clamp(st["max_norm"] / (norm + 1e-6), max=1.0).float()
    flat, views = _flat(st["grads"])
    for g, v in zip(st["grads"], views):
        v.copy_(g.float() * f)
    return dict(norm=norm.float()[None], **flat)


def _flat(grads, dtypes=(F32, BF)):
    """One buffer for all tensors of a type, as an optimiser's flat gradients, and each tensor's place in it."""
    size = [sum(g.numel() for g in grads if g.dtype == t) for t in (F32, BF)]
    flat = [torch.empty(n, dtype=t, device="cuda") for n, t in zip(size, dtypes)]
    at, views = [0, 0], []
    for g in grads:
        i = 1 if g.dtype == BF else 0
        views.append(flat[i][at[i]:at[i] + g.numel()])
        at[i] += g.numel()
    return {n: b if b.numel() else None for n, b in zip(("fp32", "bf16"), flat)}, views


PLAIN = dict(logits=_forward, head=_forward, logits_grad=_backward, head_grad=_backward, clip=_clip)


# ---------------------------------------------------------- the library's --
def _plan(st):
    """What a caller's program holds beside the inputs: descriptors, output buffers and workspaces."""
    from scale_only_quantization_amd import fqlib as F
    c, op = st["case"], st["case"]["op"]
    new = lambda dt, *shape: torch.empty(shape, dtype=dt, device="cuda")  # noqa: E731
    p = dict(F=F)
    if op == "clip":
        p["out"], views = _flat(st["grads"])
        p["list"] = F.grad_list(st["grads"], views)
        p["norm"] = new(F32, 1)
        p["ws"] = new(torch.uint8, max(8, F.grad_norm_workspace_size(p["list"])))
        return p
    T, V, m = c["T"], c["V"], c["m"]
    p["d"] = F.logprob_desc(T, V, given=m, top=c.get("k", 0), hidden=c.get("H", 0))
    if op.endswith("grad"):
        p["grad"] = new(BF, T, c["H"]) if op == "head_grad" else new(BF, T, (V + 7) // 8 * 8)[:, :V]
        size = F.head_logprob_workspace_size(p["d"], grad=True) if op == "head_grad" else 0
    else:
        k = c["k"]
        p["out"] = dict(lse=new(F32, T), entropy=new(F32, T) if c["ent"] else None, logp=new(F32, T, m) if m else None,
                        top_ids=new(torch.int32, T, k) if k else None, top_logp=new(F32, T, k) if k else None)
        size = F.head_logprob_workspace_size(p["d"]) if op == "head" else F.logprob_workspace_size(p["d"])
    p["ws"] = new(torch.uint8, size) if size else None
    return p


def _own(st):
    if "plan" not in st:
        st["plan"] = _plan(st)
    p, op = st["plan"], st["case"]["op"]
    F = p["F"]
    if op == "clip":
        F.grad_norm(p["list"], p["norm"], p["ws"])
        F.grad_clip(p["list"], st["max_norm"], p["norm"])
        return dict(norm=p["norm"], **p["out"])
    if op == "logits":
        F.logprob_fwd(p["d"], st["z"], ids=st["ids"], workspace=p["ws"], **p["out"])
        return p["out"]
    if op == "head":
        F.head_logprob_fwd(p["d"], st["h"], st["w"], ids=st["ids"], workspace=p["ws"], **p["out"])
        return p["out"]
    up = dict(ids=st["ids"], dlogp=st["dlogp"], entropy=st["entropy"], dentropy=st["dent"])
    if op == "logits_grad":
        F.logprob_bwd(p["d"], st["z"], st["lse"], p["grad"], **up)
    else:
        F.head_logprob_bwd(p["d"], st["h"], st["w"], st["lse"], p["grad"], workspace=p["ws"], **up)
    return p["grad"]


def run(state):
    return _own(state) if own else PLAIN[state["case"]["op"]](state)


# ------------------------------------------------------------------- exact --
def exact(case, seed):
    st = prepare(case, seed)
    c, op, D = case, case["op"], torch.float64
    if op == "clip":
        norm = math.sqrt(math.fsum(float(torch.dot(g.to(D), g.to(D))) for g in st["grads"]))
        f = min(1.0, st["max_norm"] / (norm + 1e-6))
        flat, views = _flat(st["grads"], (D, D))
        for g, v in zip(st["grads"], views):
            torch.mul(g.to(D), f, out=v)
        return dict(norm=torch.tensor([norm], dtype=D, device="cuda"), **flat)
    T, V, m = c["T"], c["V"], c["m"]
    w = st["w"].to(D) if "w" in st else None
    res = {}
    for r in range(0, T, 512):                                       # a few hundred rows at a time
        z = st["z"][r:r + 512].to(D) if w is None else st["h"][r:r + 512].to(D) @ w.t()
        n = z.shape[0]
        lp = torch.log_softmax(z, -1)
        p = lp.exp()
        at = torch.arange(n, device="cuda")[:, None]
        ids = st["ids"][r:r + 512].long() if m else None
        if op.endswith("grad"):
            d = torch.zeros_like(z)
            for j in range(m):
                a = torch.where(ids[:, j] >= 0, st["dlogp"][r:r + 512, j].to(D), 0.0)
                d -= a[:, None] * p
                d[at[:, 0], ids[:, j].clamp(min=0)] += a
            if c["ent"]:
                ent = -(p * lp.clamp(min=-1e300)).sum(-1, keepdim=True)
                d -= st["dent"][r:r + 512, None].to(D) * p * (lp.clamp(min=-1e300) + ent)
            part = dict(grad=d if w is None else d @ w)
        else:
            part = dict(lse=torch.logsumexp(z, -1))
            if c["ent"]:
                part["entropy"] = -(p * lp.clamp(min=-1e300)).sum(-1)
            if m:
                part["logp"] = torch.where(ids >= 0, lp[at, ids.clamp(min=0)], 0.0)
            if c["k"]:
                del p
                order = torch.cat([torch.sort(q, dim=-1, descending=True, stable=True).indices[:, :c["k"]]
                                   for q in z.split(128)])
                part["top_ids"] = order.to(torch.int32)
                part["top_logp"] = lp.gather(1, order)
        for name, v in part.items():
            res.setdefault(name, []).append(v)
    if op.endswith("grad"):
        return torch.cat(res["grad"])
    return {n: torch.cat(res[n]) if n in res else None for n in ("lse", "entropy", "logp", "top_ids", "top_logp")}
