"""The operators around the expert layer, as cases that can be timed and checked.

RMS norm with the residual's addition (forward, with 8-bit codes, backward),
the output layer's loss from hidden states (cross entropy and distillation
from a teacher's top logits, with the gradient on the hidden states), products
of packed 4-bit weights with a few rows, and the routed expert layer on packed
weights for a few tokens.  ``run`` computes them in plain torch operations in
32 bits, or, with ``own``, through the library's entry points; ``exact`` gives
the same values from the definitions in 64 bits.

Sizes are the repository's own layer (hidden 2048, expert intermediate 768,
128 experts, top-8, 16384 tokens, vocabulary 151936, top-64 of the teacher)
and generic ones.
"""
import math

import torch

own = False

EPS = 1e-6
BF = torch.bfloat16
F8 = torch.float8_e4m3fn


# ------------------------------------------------------------------- cases --
def listed():
    return [
        # one token on its way through a served model: the norm in front of an
        # FP8 layer, codes and the token's scale only (latency)
        dict(name="norm_token_fp8", op="norm", rows=1, cols=2048, residual=True, out="fp8", group=0),
        # a prompt in front of an FP8 layer with one scale per 128 elements; odd row count
        dict(name="norm_prompt_fp8", op="norm", rows=1893, cols=2048, residual=True, out="fp8", group=128),
        # a training batch (16384 tokens): bf16 output, the saved stream and 1/rms
        dict(name="norm_train", op="norm", rows=16384, cols=2048, residual=True, out="bf16", group=0),
        # its gradient, with the gradient that reaches the stream directly and d gamma
        dict(name="norm_grad", op="norm_grad", rows=16384, cols=2048, dsum=True, dgamma=True),
        # the gradient on a short ragged batch of narrow rows, frozen gamma
        dict(name="norm_grad_small", op="norm_grad", rows=77, cols=1000, dsum=False, dgamma=False),
        # the loss on a short sequence over a mid-sized vocabulary: cross entropy only, odd sizes
        dict(name="head_short_ce", op="head", T=333, H=1024, V=32003, k=0, lm=1.0, dist=0.0),
        # one sequence of a distillation step at the repository's vocabulary
        dict(name="head_sequence", op="head", T=2048, H=2048, V=151936, k=64, lm=0.8, dist=1.2),
        # the whole distillation batch (16384 tokens)
        dict(name="head_batch", op="head", T=16384, H=2048, V=151936, k=64, lm=0.8, dist=1.2),
        # one token through a dense layer's INT4 weights, one scale per 128 (latency)
        dict(name="matvec_int4", op="matvec", fmt="int4", group=128, E=1, N=2048, K=2048, M=1),
        # a few sequences' tokens through wide NVFP4 weights
        dict(name="matvec_nvfp4", op="matvec", fmt="nvfp4", group=16, E=1, N=12289, K=8192, M=13),
        # one token through the routed layer, INT4 weights (the w4a16 preset)
        dict(name="experts_token", op="experts", fmt="w4a16", E=128, H=2048, I=768, T=1, k=8),
        # sixteen sequences' tokens through it in NVFP4, activations quantised too
        dict(name="experts_tokens", op="experts", fmt="nvfp4", E=128, H=2048, I=768, T=16, k=8),
    ]


def _log(rng, lo, hi, step=1):
    v = math.exp(rng.uniform(math.log(lo), math.log(hi + 0.999)))
    return max(step, int(v) // step * step)


def draw(rng):
    op = rng.choice(["norm", "norm", "norm_grad", "head", "head", "matvec", "experts"])
    if op == "norm":
        out = rng.choice(["bf16", "fp8", "both"])
        group = rng.choice([0, 64, 128]) if out != "bf16" else 0
        cols = _log(rng, 128, 8192, group or 8)
        return dict(op=op, rows=_log(rng, 1, min(16384, 4_000_000 // cols)), cols=cols,
                    residual=rng.random() < 0.7, out=out, group=group)
    if op == "norm_grad":
        return dict(op=op, rows=_log(rng, 1, 16384), cols=_log(rng, 128, 8192, 8), dsum=rng.random() < 0.5,
                    dgamma=rng.random() < 0.5)
    if op == "head":
        k = rng.choice([0, 1, 16, 33, 64])
        return dict(op=op, T=_log(rng, 1, 4096), H=_log(rng, 128, 4096, 64), V=_log(rng, 1000, 151936), k=k,
                    lm=1.0 if k == 0 else rng.choice([0.0, 0.5, 1.0]), dist=rng.choice([0.5, 1.0]))
    if op == "matvec":
        fmt = rng.choice(["int4", "nvfp4"])
        group = rng.choice([32, 64, 128]) if fmt == "int4" else 16
        E = rng.choice([1, 1, 4])
        return dict(op=op, fmt=fmt, group=group, E=E, N=_log(rng, 64, 12289), K=_log(rng, 128, 8192, 128),
                    M=_log(rng, 1, 48))
    E = rng.choice([8, 32, 128])
    return dict(op=op, fmt=rng.choice(["w4a16", "nvfp4", "nvfp4a16", "w4afp8"]), E=E, H=_log(rng, 256, 2048, 128),
                I=_log(rng, 128, 1024, 128), T=_log(rng, 1, 32), k=rng.choice([1, 2, 4, 8]))


def work(case):
    c, op = case, case["op"]
    if op == "norm":
        n = c["rows"] * c["cols"]
        b = 2 * n * (1 + 2 * c["residual"]) + 2 * c["cols"]
        b += 2 * n if c["out"] != "fp8" else 0
        b += n + 4 * c["rows"] * (c["cols"] // c["group"] if c["group"] else 1) if c["out"] != "bf16" else 0
        return dict(bytes=b + 4 * c["rows"], flops=4 * n)
    if op == "norm_grad":
        n = c["rows"] * c["cols"]
        return dict(bytes=2 * n * (3 + c["dsum"]) + 4 * c["rows"] + 2 * c["cols"] + 4 * c["cols"] * c["dgamma"],
                    flops=8 * n)
    if op == "head":
        T, H, V = c["T"], c["H"], c["V"]
        return dict(bytes=2 * V * H + 4 * T * H + T * (8 + 8 * c["k"]), flops=4 * T * V * H)
    if op == "matvec":
        E = min(c["E"], c["M"])
        per = 4 / c["group"] if c["fmt"] == "int4" else 1 / 16
        return dict(bytes=E * c["N"] * c["K"] * (0.5 + per) + 2 * c["M"] * (c["N"] + c["K"]),
                    flops=2 * c["M"] * c["N"] * c["K"])
    hit = c["E"] * (1 - (1 - c["k"] / c["E"]) ** c["T"])              # experts hit by uniform routing
    per = 4 / 128 if c["fmt"] in ("w4a16", "w4afp8") else 1 / 16
    n = 3 * c["H"] * c["I"]
    return dict(bytes=hit * n * (0.5 + per) + 4 * c["T"] * c["H"], flops=2 * c["T"] * c["k"] * n)


# ------------------------------------------------------------------ inputs --
def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _randn(g, *shape):
    return torch.randn(shape, generator=g, device="cuda")


def _pack(q):
    """4-bit codes [..., K] (uint8) packed two per byte, the even column in the low nibble."""
    return (q[..., 0::2] | (q[..., 1::2] << 4)).contiguous()


def _pack_int4(W, group):
    """INT4 [-8, 7] codes of W [E, N, K] and one fp32 scale per `group` columns."""
    E, N, K = W.shape
    b = W.view(E, N, K // group, group)
    s = b.abs().amax(-1) / 7.0
    q = torch.round(b / s[..., None]).clamp_(-8, 7).to(torch.int8).view(torch.uint8) & 15
    return dict(codes=_pack(q.view(E, N, K)), scale=s.contiguous())


def _pack_nvfp4(W):
    """E2M1 codes of W [E, N, K], E4M3 block factors per 16 columns (bytes) and a tensor scale per matrix."""
    E, N, K = W.shape
    t = W.abs().amax((1, 2)) / 2688.0
    b = W.view(E, N, K // 16, 16)
    d = (b.abs().amax(-1) / 6.0 / t[:, None, None]).clamp(max=448.0).to(F8)
    s = d.float() * t[:, None, None]
    a = (b.abs() / s.clamp(min=1e-30)[..., None])
    q = torch.zeros_like(a, dtype=torch.uint8)
    for mid in (0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0):
        q += a > mid
    q |= (b < 0).to(torch.uint8) << 3
    return dict(codes=_pack(q.view(E, N, K)), block_codes=d.view(torch.uint8).contiguous(), tensor_scale=t)


def _weights(g, fmt, group, E, N, K):
    W = _randn(g, E, N, K) * 0.02
    return _pack_int4(W, group) if fmt == "int4" else _pack_nvfp4(W)


def prepare(case, seed):
    g, c, op = _gen(seed), case, case["op"]
    s = dict(case=c)
    if op in ("norm", "norm_grad"):
        R, C = c["rows"], c["cols"]
        s["gamma"] = (1.0 + 0.2 * _randn(g, C)).to(BF)
        size = torch.exp(0.5 * _randn(g, R, 1))                      # tokens of different magnitude
        x = (_randn(g, R, C) * size).to(BF)
        if op == "norm":
            s["x"] = x
            s["res"] = (_randn(g, R, C) * 2.0 * size).to(BF) if c["residual"] else None
        else:
            s["s"] = x
            s["rstd"] = torch.rsqrt(x.double().square().mean(-1) + EPS).float()
            s["dy"] = (_randn(g, R, C) * 0.01).to(BF)
            s["dsum"] = (_randn(g, R, C) * 0.01).to(BF) if c["dsum"] else None
    elif op == "head":
        T, H, V, k = c["T"], c["H"], c["V"], c["k"]
        w = (_randn(g, V, H) * (2.0 / math.sqrt(H))).to(BF)          # logits of standard deviation 2
        labels = torch.randint(0, V, (T,), generator=g, device="cuda")
        sure = torch.rand((T, 1), generator=g, device="cuda") * 12.0  # how much the label's logit stands out
        h = _randn(g, T, H) + sure / 4.0 * w[labels].float()
        labels[torch.rand((T,), generator=g, device="cuda") < 0.05] = -1   # padding
        if T == 1:
            labels.clamp_(min=0)
        s.update(h=h.to(BF), w=w, labels=labels.to(torch.int32) if c["lm"] else None, tv=None, ti=None)
        if k:
            tv, ti = [], []
            for r in range(0, T, 2048):                              # the teacher: the same model, other numerics
                z = (h[r:r + 2048] + 0.3 * _randn(g, *h[r:r + 2048].shape)).to(BF) @ w.t()
                v, i = torch.topk(z.float(), k, dim=-1)
                tv.append(v)
                ti.append(i.to(torch.int32))
            s.update(tv=torch.cat(tv), ti=torch.cat(ti))
    elif op == "matvec":
        s.update(_weights(g, c["fmt"], c["group"], c["E"], c["N"], c["K"]))
        s["x"] = _randn(g, c["M"], c["K"]).to(BF)
        s["which"] = (torch.randint(0, c["E"], (c["M"],), generator=g, device="cuda").to(torch.int32)
                      if c["E"] > 1 else None)
    else:
        E, H, I, T, k = (c[n] for n in ("E", "H", "I", "T", "k"))
        fmt = "int4" if c["fmt"] in ("w4a16", "w4afp8") else "nvfp4"
        s["w1"] = _weights(g, fmt, 128, E, 2 * I, H)
        s["w2"] = _weights(g, fmt, 128, E, H, I)
        s["x"] = _randn(g, T, H).to(BF)
        s["ids"] = torch.rand((T, E), generator=g, device="cuda").topk(k, -1).indices.to(torch.int32)
        s["tw"] = torch.softmax(_randn(g, T, k), -1)
        div = {"nvfp4": 2688.0, "w4afp8": 448.0}.get(c["fmt"])
        u = 0.9 + 0.2 * torch.rand((E,), generator=g, device="cuda")
        s["s_a1"] = 4.5 / div * u if div else None
        s["s_a2"] = 6.0 * H / 2048 / div * u if div else None
    return s


# -------------------------------------------------------------- plain forms --
# Every function takes the type its arithmetic runs in: 32 bits for the plain
# forms, 64 for `exact`'s building blocks that are one operation each.
def _nibbles(codes):
    return torch.stack((codes & 15, codes >> 4), -1).flatten(-2)


def _dequant(w, pick, ft):
    """Matrices `pick` (an index tensor, or a slice) of packed weights, as [n, N, K] in type ft."""
    q = _nibbles(w["codes"][pick])
    if "scale" in w:
        v = (((q ^ 8).to(ft)) - 8)
        sc = w["scale"][pick].to(ft)
    else:
        tab = torch.tensor([0, 0.5, 1, 1.5, 2, 3, 4, 6, -0.0, -0.5, -1, -1.5, -2, -3, -4, -6], device="cuda", dtype=ft)
        v = tab[q.int()]
        sc = w["block_codes"].view(F8)[pick].to(ft) * w["tensor_scale"][pick].to(ft)[:, None, None]
    n, N, K = v.shape
    return (v.view(n, N, sc.shape[-1], -1) * sc[..., None]).view(n, N, K)


def _fake_quant(x, fmt, s):
    """The layer's activation quantisers on bf16 rows x [R, K], s [R] the scale of each row's expert; bf16 values."""
    if s is None:
        return x
    f = x.float()
    if fmt == "w4afp8":
        sh = s[:, None]
        q = (f / sh).clamp(-448.0, 448.0).to(F8).float()
    else:
        b = f.view(f.shape[0], -1, 16)
        sh = s[:, None] * (b.abs().amax(-1) / (6.0 * s[:, None])).clamp(max=448.0).to(F8).float()
        sh = sh.repeat_interleave(16, -1)
        r = torch.where(sh > 0, f / sh, torch.zeros_like(f))
        a = r.abs().clamp(max=6.0)
        step = torch.where(a < 2, 0.5, torch.where(a < 4, 1.0, 2.0))
        q = torch.copysign(torch.round(a / step) * step, f)
    return (q * sh).to(BF)


def _quant8(y, group):
    """E4M3 values and scales of bf16 y, one scale per row or per `group` columns."""
    f = y.float()
    b = f.view(f.shape[0], -1, group) if group else f[:, None, :]
    s = b.abs().amax(-1) / 448.0
    q = torch.where(s[..., None] > 0, b / s[..., None], torch.zeros_like(b)).clamp(-448.0, 448.0).to(F8)
    return q.view_as(f), s if group else s[:, 0]


def _norm(st, ft):
    c = st["case"]
    x = st["x"]
    out = {}
    if st["res"] is not None:
        x = (x.to(ft) + st["res"].to(ft)).to(BF)
        out["sum"] = x
    # 64 bits up to y: a bf16 value on the other side of a rounding border
    # would move a whole group's scale
    f = x.double()
    rstd = 1.0 / torch.sqrt((f * f).mean(-1) + EPS)
    y = (f * st["gamma"].double() * rstd[:, None]).float().to(BF)
    out["rstd"] = rstd.to(ft)
    if c["out"] != "fp8":
        out["y"] = y
    if c["out"] != "bf16":
        out["codes"], out["scale"] = _quant8(y, c["group"])
    return out


def _norm_grad(st, ft):
    s, rstd, g, dy = st["s"].to(ft), st["rstd"].to(ft)[:, None], st["gamma"].to(ft), st["dy"].to(ft)
    a = dy * g
    dx = rstd * (a - s * (rstd * rstd * (a * s).mean(-1, keepdim=True)))
    if st["dsum"] is not None:
        dx = dx + st["dsum"].to(ft)
    return dict(dx=dx.to(BF) if ft == torch.float32 else dx,
                dgamma=(dy * s * rstd).sum(0) if st["case"]["dgamma"] else None)


def _head(st, ft):
    c, w, lab, tv, ti = st["case"], st["w"].to(ft), st["labels"], st["tv"], st["ti"]
    T = c["T"]
    z = st["h"].to(ft) @ w.t()
    lse = torch.logsumexp(z, -1) if ft == torch.float64 else None
    if lse is None:
        m = z.amax(-1)
        lse = m + torch.log(torch.exp(z - m[:, None]).sum(-1))
    live = torch.ones(T, dtype=torch.bool, device="cuda") if lab is None else lab >= 0
    n = live.sum().clamp(min=1).to(ft)
    rows = torch.zeros(T, device="cuda", dtype=ft)
    wq = 0.0
    if lab is not None:
        at = lab.long().clamp(min=0)[:, None]
        rows = rows + c["lm"] * (lse - z.gather(1, at)[:, 0])
        wq += c["lm"]
    if tv is not None:
        t = tv.to(ft)
        lp = t - t.amax(-1, keepdim=True)
        lp = lp - torch.log(torch.exp(lp).sum(-1, keepdim=True))
        p = torch.exp(lp)
        rows = rows + c["dist"] * (p * (lp - z.gather(1, ti.long()) + lse[:, None])).sum(-1)
        wq += c["dist"]
    z.sub_(lse[:, None]).exp_().mul_(wq)                             # now d rows / d z
    if lab is not None:
        z.scatter_add_(1, at, torch.full_like(at, -c["lm"], dtype=ft))
    if tv is not None:
        z.scatter_add_(1, ti.long(), -c["dist"] * p)
    rows = torch.where(live, rows, torch.zeros_like(rows))
    grad = (z @ w) * (live.to(ft) / n)[:, None]
    return dict(loss=rows.sum()[None] / n, rows=rows, grad=grad.to(BF) if ft == torch.float32 else grad)


def _matvec(st, ft):
    x, which = st["x"].to(ft), st["which"]
    if which is None:
        y = x @ _dequant(st, slice(0, 1), ft)[0].t()
    else:
        y = torch.matmul(_dequant(st, slice(None), ft)[which.long()], x[:, :, None])[:, :, 0]
    return y.to(BF) if ft == torch.float32 else y


def _experts(st, ft):
    c, k = st["case"], st["case"]["k"]
    e = st["ids"].long().flatten()
    pick = lambda v: None if v is None else v[e]  # noqa: E731
    x = _fake_quant(st["x"].repeat_interleave(k, 0), c["fmt"], pick(st["s_a1"])).to(ft)
    z = torch.matmul(_dequant(st["w1"], e, ft), x[:, :, None])[:, :, 0]
    gate, up = z[:, :c["I"]], z[:, c["I"]:]
    h = _fake_quant((gate / (1.0 + torch.exp(-gate)) * up).to(BF), c["fmt"], pick(st["s_a2"])).to(ft)
    y = torch.matmul(_dequant(st["w2"], e, ft), h[:, :, None])[:, :, 0]
    y = (y.view(c["T"], k, -1) * st["tw"].to(ft)[..., None]).sum(1)
    return y.to(BF) if ft == torch.float32 else y


PLAIN = dict(norm=_norm, norm_grad=_norm_grad, head=_head, matvec=_matvec, experts=_experts)


# ---------------------------------------------------------- the library's --
def _plan(st):
    """What a caller's program holds beside the inputs: descriptors, output buffers and workspaces."""
    from scale_only_quantization_amd import fqlib as F
    c, op = st["case"], st["case"]["op"]
    new = lambda dt, *shape: torch.empty(shape, dtype=dt, device="cuda")  # noqa: E731
    p = dict(F=F)
    if op == "norm":
        R, C, g = c["rows"], c["cols"], c["group"]
        p["sum"] = new(BF, R, C) if c["residual"] else None
        p["y"] = new(BF, R, C) if c["out"] != "fp8" else None
        p["rstd"] = new(torch.float32, R)
        p["q"] = p["codes"] = p["scale"] = None
        if c["out"] != "bf16":
            p["q"] = F.qdesc(F.FQ_FP8E4M3, F.FQ_PER_GROUP if g else F.FQ_PER_ROW, g, F.FQ_DYNAMIC)
            p["codes"] = new(torch.uint8, R, C)
            p["scale"] = new(torch.float32, R, C // g) if g else new(torch.float32, R)
    elif op == "norm_grad":
        R, C = c["rows"], c["cols"]
        p["dx"] = new(BF, R, C)
        p["dgamma"] = new(torch.float32, C) if c["dgamma"] else None
        p["ws"] = new(torch.uint8, max(16, F.rms_norm_bwd_workspace_size(R, C))) if c["dgamma"] else None
    elif op == "head":
        p["d"] = F.head_desc(c["T"], c["H"], c["V"], c["k"], c["lm"], c["dist"])
        p["loss"], p["rows"] = new(torch.float32, 1), new(torch.float32, c["T"])
        p["grad"] = new(BF, c["T"], c["H"])
        p["ws"] = new(torch.uint8, F.head_loss_workspace_size(p["d"]))
    elif op == "matvec":
        p["q"] = (F.qdesc(F.FQ_INT, F.FQ_PER_GROUP, c["group"], F.FQ_LEARNABLE, -8, 7) if c["fmt"] == "int4"
                  else F.qdesc(F.FQ_NVFP4, F.FQ_PER_GROUP, 16, F.FQ_LEARNABLE))
        p["y"] = new(BF, c["M"], c["N"])
    else:
        p["L"] = F.layer_desc(c["E"], c["H"], c["I"], c["T"], c["k"], *F.preset(c["fmt"]))
        p["P"] = F.packed_experts(st["w1"], st["w2"], st["s_a1"], st["s_a2"])
        p["y"] = new(BF, c["T"], c["H"])
        p["ws"] = new(torch.uint8, F.packed_expert_workspace_size(p["L"]))
    return p


def _own(st):
    if "plan" not in st:
        st["plan"] = _plan(st)
    p, op = st["plan"], st["case"]["op"]
    F = p["F"]
    if op == "norm":
        F.rms_norm_fwd(st["x"], st["gamma"], EPS, residual=st["res"], sum=p["sum"], y=p["y"], rstd=p["rstd"],
                       q=p["q"], codes=p["codes"], scale=p["scale"])
        out = dict(sum=p["sum"], rstd=p["rstd"], y=p["y"])
        if p["codes"] is not None:
            out.update(codes=p["codes"].view(F8), scale=p["scale"])
        return out
    if op == "norm_grad":
        F.rms_norm_bwd(st["s"], st["gamma"], st["rstd"], st["dy"], p["dx"], dsum=st["dsum"], dgamma=p["dgamma"],
                       workspace=p["ws"])
        return dict(dx=p["dx"], dgamma=p["dgamma"])
    if op == "head":
        F.head_loss(p["d"], st["h"], st["w"], p["loss"], top_v=st["tv"], top_i=st["ti"], labels=st["labels"],
                    row_loss=p["rows"], grad=p["grad"], workspace=p["ws"])
        return dict(loss=p["loss"], rows=p["rows"], grad=p["grad"])
    if op == "matvec":
        F.packed_matvec(p["q"], st["codes"], st["x"], p["y"], scale=st.get("scale"),
                        block_codes=st.get("block_codes"), tensor_scale=st.get("tensor_scale"), which=st["which"])
        return p["y"]
    F.packed_expert_fwd(p["L"], p["P"], st["x"], st["ids"], st["tw"], p["y"], p["ws"])
    return p["y"]


def run(state):
    return _own(state) if own else PLAIN[state["case"]["op"]](state, torch.float32)


# ------------------------------------------------------------------- exact --
def exact(case, seed):
    st = prepare(case, seed)
    op, D = case["op"], torch.float64
    if op == "norm":
        x = st["x"].to(D) if st["res"] is None else (st["x"].to(D) + st["res"].to(D)).to(BF).to(D)
        r = (x.square().sum(-1) / case["cols"] + EPS).pow(-0.5)
        y = (x * (r[:, None] * st["gamma"].to(D))).float().to(BF)    # the norm's bf16 output is what is quantised
        out = dict(rstd=r, y=y.to(D) if case["out"] != "fp8" else None,
                   sum=x if st["res"] is not None else None)
        if case["out"] != "bf16":
            b = y.to(D).view(case["rows"], -1, case["group"] or case["cols"])
            s = b.abs().amax(-1) / 448.0
            q = (b / s.clamp(min=1e-300)[..., None]).clamp(-448, 448).to(F8).to(D).view_as(y)
            out.update(codes=q, scale=s if case["group"] else s[:, 0])
        return out
    if op == "norm_grad":
        s, r, g, dy = st["s"].to(D), st["rstd"].to(D), st["gamma"].to(D), st["dy"].to(D)
        n = s * r[:, None]
        along = (dy * g * n).sum(-1) / case["cols"]
        dx = (dy * g - n * along[:, None]) * r[:, None]
        if st["dsum"] is not None:
            dx += st["dsum"].to(D)
        return dict(dx=dx, dgamma=torch.einsum("tc,tc->c", dy, n) if case["dgamma"] else None)
    if op == "head":
        w, lab = st["w"].to(D), st["labels"]
        T = case["T"]
        rows = torch.zeros(T, device="cuda", dtype=D)
        grad = torch.zeros((T, case["H"]), device="cuda", dtype=D)
        keep = torch.arange(T, device="cuda") if lab is None else torch.nonzero(lab >= 0)[:, 0]
        n = max(1, keep.numel())
        for part in keep.split(4096):                                # rows that count, a few thousand at a time
            lq = torch.log_softmax(st["h"][part].to(D) @ w.t(), -1)
            g = torch.zeros_like(lq)
            if lab is not None:
                at = (torch.arange(part.numel(), device="cuda"), lab[part].long())
                rows[part] -= case["lm"] * lq[at]
                g += case["lm"] * lq.exp()
                g[at] -= case["lm"]
            if st["tv"] is not None:
                lp = torch.log_softmax(st["tv"][part].to(D), -1)
                ti = st["ti"][part].long()
                rows[part] += case["dist"] * (lp.exp() * (lp - lq.gather(1, ti))).sum(-1)
                g += case["dist"] * lq.exp()
                g.scatter_add_(1, ti, -case["dist"] * lp.exp())
            grad[part] = g @ w / n
        return dict(loss=rows.sum()[None] / n, rows=rows, grad=grad)
    if op == "matvec":
        x = st["x"].to(D)
        y = torch.empty((case["M"], case["N"]), device="cuda", dtype=D)
        for m in range(case["M"]):                                   # row by row
            e = 0 if st["which"] is None else int(st["which"][m])
            y[m] = _dequant(st, slice(e, e + 1), D)[0] @ x[m]
        return y
    y = torch.zeros((case["T"], case["H"]), device="cuda", dtype=D)
    I = case["I"]
    for t in range(case["T"]):                                       # token by token, slot by slot
        for j in range(case["k"]):
            e = int(st["ids"][t, j])
            one = slice(e, e + 1)
            sc = [None if st[n] is None else st[n][one] for n in ("s_a1", "s_a2")]
            x = _fake_quant(st["x"][t:t + 1], case["fmt"], sc[0])[0].to(D)
            z = _dequant(st["w1"], one, D)[0] @ x
            h = (z[:I] * torch.sigmoid(z[:I]) * z[I:]).to(BF)
            h = _fake_quant(h[None], case["fmt"], sc[1])[0].to(D)
            y[t] += st["tw"][t, j].to(D) * (_dequant(st["w2"], one, D)[0] @ h)
    return y
