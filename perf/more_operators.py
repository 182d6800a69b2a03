"""Measured cases of the training head's operators: the layer norm before the LM
head (layer_norm), its backward pass (layer_norm_backward) and the gradient of the
fused linear + logprob (linear_logp_backward), with a plain form of each.

Layer norm. y = (x - m) r w + b over each row, with m the mean (0 for the RMS
form) and r = 1 / sqrt(mean((x - m)^2) + eps). The backward pass takes the
forward's m and r and returns the gradients of x, w and b.

Linear + logprob. x_ij = bf16(sum_k h_ik w_jk), z = x / T. Each row's loss is
g_r times the logprob of its target over the whole vocabulary plus g_p times the
logprob over the support (x >= threshold). Given the forward call's statistics,
the gradients of the hidden states and of the projection are returned; the
logits are not kept between the two calls.
"""
import math

import torch

own = False

HEAD_REAL, HEAD_PADDED, HEAD_D = 151936, 152576, 4096  # the benchmark's vocabulary and hidden width
EPS = 1e-6


def listed():
    head = dict(d=HEAD_D, vocab_real=HEAD_REAL, vocab_padded=HEAD_PADDED)
    return [
        # one decoded token: latency
        dict(name="norm 1 x 4096", op="norm", rows=1, d=HEAD_D, rms=True, bias=False, x32=False, w32=False, pad=0),
        # an odd row count out of a wider buffer, with a bias
        dict(name="norm 4999 x 2080 strided", op="norm", rows=4999, d=2080, rms=False, bias=True, x32=False, w32=True, pad=96),
        # a training batch whose residual stream is kept in 32 bits
        dict(name="norm 8192 x 4096 fp32", op="norm", rows=8192, d=HEAD_D, rms=True, bias=False, x32=True, w32=False, pad=0),
        # a small model's odd batch
        dict(name="norm backward 37 x 1000", op="norm backward", rows=37, d=1000, rms=False, bias=True, x32=True, w32=True, pad=8),
        # a training batch
        dict(name="norm backward 8192 x 4096", op="norm backward", rows=8192, d=HEAD_D, rms=True, bias=False, x32=False, w32=False, pad=0),
        # long sequences packed into one batch
        dict(name="norm backward 65536 x 4096", op="norm backward", rows=65536, d=HEAD_D, rms=False, bias=True, x32=False, w32=False, pad=0),
        # one token: an online update
        dict(name="grad 1", op="grad", rows=1, terms="ref", temperature=1.0, masked=0.0, wants="both", **head),
        # a short answer, both logprobs in the loss
        dict(name="grad 48 both terms", op="grad", rows=48, terms="both", temperature=0.7, masked=0.0, wants="both", **head),
        # odd sizes throughout, temperatures per request, greedy ones among them
        dict(name="grad 77 x 1088 x 50021", op="grad", rows=77, d=1088, vocab_real=50021, vocab_padded=50048, terms="ref", temperature=-1.0,
             masked=0.0, wants="both"),
        # a frozen head: hidden states' gradient alone
        dict(name="grad 640 hidden", op="grad", rows=640, terms="ref", temperature=1.0, masked=0.0, wants="hidden", **head),
        # prompts and answers: half of the rows carry no loss
        dict(name="grad 3000 half masked", op="grad", rows=3000, terms="ref", temperature=1.0, masked=0.5, wants="both", **head),
        # a training step's 8192 tokens
        dict(name="grad 8192", op="grad", rows=8192, terms="ref", temperature=0.7, masked=0.0, wants="both", **head),
    ]


def _between(rng, lo, hi):
    """A whole number in [lo, hi], spread over its logarithm."""
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["norm", "norm backward", "grad", "grad"])
    if op != "grad":
        d = 8 * _between(rng, 1, 1024)
        return dict(op=op, rows=_between(rng, 1, min(65536, (1 << 27) // d)), d=d, rms=rng.random() < 0.5, bias=rng.random() < 0.5,
                    x32=rng.random() < 0.4, w32=rng.random() < 0.4, pad=rng.choice([0, 0, 8, 96]))
    if rng.random() < 0.4:
        real, padded = HEAD_REAL, HEAD_PADDED
    else:
        real = _between(rng, 300, HEAD_REAL)
        padded = (real + 63) // 64 * 64 + 64 * rng.choice([0, 0, 1, 5])
    terms = rng.choice(["ref", "ref", "both", "policy"])
    return dict(op=op, rows=_between(rng, 1, 4096 if terms == "ref" else 256), d=64 * _between(rng, 1, HEAD_D // 64), vocab_real=real,
                vocab_padded=padded, terms=terms, temperature=rng.choice([1.0, 0.7, 1.3, -1.0]), masked=rng.choice([0.0, 0.0, 0.3, 0.7]),
                wants=rng.choice(["both", "both", "hidden", "weight"]))


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------

def _prepare_norm(c, gen, dev):
    n, d = c["rows"], c["d"]
    xt, wt = (torch.float32 if c[k] else torch.bfloat16 for k in ("x32", "w32"))
    x = torch.empty((n, d + c["pad"]), dtype=xt, device=dev)
    x.normal_(generator=gen)
    # rows of unlike magnitude, a common offset, and a few channels that are much larger than the rest
    x *= torch.exp2(torch.randint(-2, 3, (n, 1), generator=gen, device=dev).float()).to(xt)
    x += 0.25
    x[:, ::max(1, d // 5)] *= 20
    x = x[:, :d]
    w = (1 + 0.2 * torch.randn(d, generator=gen, device=dev)).to(wt)
    b = (0.1 * torch.randn(d, generator=gen, device=dev)).to(wt) if c["bias"] else None
    s = dict(op=c["op"], rms=c["rms"], x=x, w=w, b=b)
    if c["op"] == "norm backward":
        mean, var = torch.empty(n, device=dev), torch.empty(n, device=dev)
        for at in range(0, n, 8192):
            v = x[at:at + 8192].double()
            m = torch.zeros_like(v[:, 0]) if c["rms"] else v.mean(1)
            mean[at:at + 8192] = m.float()
            var[at:at + 8192] = (v - m[:, None]).square().mean(1).float()
        s["mean"], s["rstd"] = mean, 1 / torch.sqrt(var + EPS)
        s["dy"] = (torch.randn((n, d), generator=gen, device=dev, dtype=torch.bfloat16) * (1.0 / n))
    return s


def _prepare_grad(c, gen, dev):
    n, d, real, padded = c["rows"], c["d"], c["vocab_real"], c["vocab_padded"]
    w = torch.empty((real, d), dtype=torch.bfloat16, device=dev).normal_(generator=gen)
    w *= 2.5 / math.sqrt(d)
    target = torch.randint(0, real, (n,), generator=gen, device=dev)
    # normed hidden states that lean towards their target: its logit is raised by 0 to 15
    lean = torch.rand((n, 1), generator=gen, device=dev) * 2.4
    h = (torch.randn((n, d), generator=gen, device=dev) + lean * w[target].float()).to(torch.bfloat16)
    if c["temperature"] < 0:  # per request, greedy ones among them
        t = torch.tensor([0.7, 1.0, 1.3, 0.0], device=dev)[torch.randint(0, 4, (n,), generator=gen, device=dev)]
    else:
        t = torch.full((n,), c["temperature"], device=dev)
    ref, pol, lse = (torch.empty(n, device=dev) for _ in range(3))
    state = torch.zeros((n, 4), dtype=torch.int32, device=dev)
    wf, step = w.float(), 1024 if c["terms"] == "ref" else 64
    for at in range(0, n, step):  # what the forward call leaves of each row
        here = slice(at, at + step)
        x = (h[here].float() @ wf.T).to(torch.bfloat16)
        greedy = t[here, None] == 0
        z = x.float() / torch.where(greedy, 1.0, t[here, None])
        full = torch.logsumexp(z, 1, keepdim=True)
        zt = torch.gather(z, 1, target[here, None])
        point = torch.where(torch.argmax(x, 1, keepdim=True) == target[here, None], 0.0, -math.inf)
        ref[here] = torch.where(greedy, point, zt - full)[:, 0]
        lse[here] = torch.where(greedy, math.nan, full)[:, 0]
        if c["terms"] != "ref":  # the support that holds 0.95 of the mass
            order = torch.sort(z, 1, descending=True).values
            last = (torch.cumsum(torch.exp((order - full).double()), 1) < 0.95).sum(1, keepdim=True).clamp(max=real - 1)
            kept = z >= torch.gather(order, 1, last)
            part = torch.logsumexp(torch.where(kept, z, -math.inf), 1, keepdim=True)
            hit = torch.where(greedy, point == 0, torch.gather(kept, 1, target[here, None]))
            pol[here] = torch.where(greedy, point, torch.where(hit, zt - part, -math.inf))[:, 0]
            state[here, 0] = torch.where(greedy, math.nan, part)[:, 0].view(torch.int32)
            state[here, 1] = torch.where(greedy, -math.inf, torch.where(kept, x.float(), math.inf).amin(1, keepdim=True))[:, 0].view(torch.int32)
            state[here, 2] = hit[:, 0].int()
    carries = torch.ones(n, device=dev)
    carries[torch.randperm(n, generator=gen, device=dev)[:n - _active(c)]] = 0
    g = torch.randn((2, n), generator=gen, device=dev) / max(1, _active(c)) * carries
    return dict(op="grad", h=h, w=w, t=t, target=target, padded=padded, wants=c["wants"], ref=ref, lse=lse, pol=pol, state=state,
                g_ref=g[0].contiguous() if c["terms"] != "policy" else None, g_pol=g[1].contiguous() if c["terms"] != "ref" else None)


def _active(c):
    """Rows that carry a loss."""
    return max(1, c["rows"] - int(c["masked"] * c["rows"]))


def prepare(case, seed):
    dev = torch.device("cuda:0")
    gen = torch.Generator(device=dev)
    gen.manual_seed(seed)
    return (_prepare_grad if case["op"] == "grad" else _prepare_norm)(case, gen, dev)


# ---------------------------------------------------------------------------
# the operators: the framework's calls and their plain forms
# ---------------------------------------------------------------------------

def run(s):
    if own:
        return _call(s)
    return {"norm": _plain_norm, "norm backward": _plain_norm_backward, "grad": _plain_grad}[s["op"]](s)


def _call(s):
    import invariant_token_log_fp32_amd as rlk
    if s["op"] == "norm":
        y, mean, rstd = rlk.layer_norm(s["x"], s["w"], s["b"], rms=s["rms"], eps=EPS, return_stats=True)
        return (y, rstd) if s["rms"] else (y, mean, rstd)
    if s["op"] == "norm backward":
        dx, dw, db = rlk.layer_norm_backward(s["dy"], s["x"], s["w"], None if s["rms"] else s["mean"], s["rstd"], rms=s["rms"],
                                             bias_grad=s["b"] is not None)
        return (dx, dw) if db is None else (dx, dw, db)
    dh, dw = rlk.linear_logp_backward(s["h"], s["w"], s["t"], s["target"], vocab_padded=s["padded"], ref_logp=s["ref"], lse=s["lse"],
                                      grad_ref=s["g_ref"], policy_logp=s["pol"], support_state=s["state"], grad_policy=s["g_pol"],
                                      hidden_grad=s["wants"] != "weight", weight_grad=s["wants"] != "hidden")
    return [v for v in (dh, dw) if v is not None]


def _plain_norm(s):
    x = s["x"].float()
    mean = torch.zeros_like(x[:, :1]) if s["rms"] else x.mean(1, keepdim=True)
    rstd = 1 / torch.sqrt((x - mean).square().mean(1, keepdim=True) + EPS)
    y = (x - mean) * rstd * s["w"].float()
    if s["b"] is not None:
        y = y + s["b"].float()
    y = y.to(torch.bfloat16)
    return (y, rstd[:, 0]) if s["rms"] else (y, mean[:, 0], rstd[:, 0])


def _plain_norm_backward(s):
    x, dy = s["x"].float(), s["dy"].float()
    r = s["rstd"][:, None]
    hat = x * r if s["rms"] else (x - s["mean"][:, None]) * r
    g = dy * s["w"].float()
    dx = g - hat * (g * hat).mean(1, keepdim=True)
    if not s["rms"]:
        dx = dx - g.mean(1, keepdim=True)
    out = ((dx * r).to(s["x"].dtype), (dy * hat).sum(0))
    return out if s["b"] is None else out + (dy.sum(0),)


def _plain_grad(s):
    # the logits are rounded to BF16 by definition, so a sum next to the middle of two
    # values has to be right: 64 bits
    x = (s["h"].double() @ s["w"].double().T).to(torch.bfloat16).float()
    t = s["t"][:, None]
    live = t > 0
    safe = torch.where(live, t, 1.0)
    z, g, at = x / safe, torch.zeros_like(x), torch.zeros_like(t)
    if s["g_ref"] is not None:
        up = s["g_ref"][:, None]
        g = g - up * torch.exp(z - s["lse"][:, None])
        at = at - up * torch.expm1(s["ref"][:, None])
    if s["g_pol"] is not None:
        part, threshold, hit = s["state"][:, 0:1].view(torch.float32), s["state"][:, 1:2].view(torch.float32), s["state"][:, 2:3] == 1
        up = torch.where(hit, s["g_pol"][:, None], 0.0)
        g = g - up * torch.where(x >= threshold, torch.exp(z - part), 0.0)
        at = at - up * torch.where(hit, torch.expm1(s["pol"][:, None]), 0.0)
    g = torch.where(live, g.scatter(1, s["target"][:, None], at) / safe, 0.0)
    out = []
    if s["wants"] != "weight":
        out.append((g @ s["w"].float()).to(torch.bfloat16))
    if s["wants"] != "hidden":
        out.append((g.T @ s["h"].float()).to(torch.bfloat16))
    return out


# ---------------------------------------------------------------------------
# what a pass cannot do without, and what it returns in 64 bits
# ---------------------------------------------------------------------------

def work(case):
    c = case
    n, d = c["rows"], c["d"]
    if c["op"] != "grad":
        sx, sw = 4 if c["x32"] else 2, 4 if c["w32"] else 2
        back, vectors = c["op"] == "norm backward", 2 if c["bias"] else 1
        if back:
            return {"bytes": n * d * (2 + 2 * sx) + n * 8 + d * (sw + 4 * vectors), "flops": 12 * n * d}
        return {"bytes": n * d * (sx + 2) + n * 8 + d * sw * vectors, "flops": 8 * n * d}
    real, live = c["vocab_real"], _active(c)
    products = 1 + (c["wants"] != "weight") + (c["wants"] != "hidden")
    moved = live * d + real * d + (n * d if c["wants"] != "weight" else 0) + (real * d if c["wants"] != "hidden" else 0)
    return {"bytes": 2 * moved + 40 * n, "flops": 2 * products * live * real * d}


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "grad":
        return _exact_grad(s)
    x, w = s["x"].double(), s["w"].double()
    n, d = x.shape
    if case["op"] == "norm":
        mean = x.new_zeros(n) if case["rms"] else x.sum(1) / d
        x -= mean[:, None]
        rstd = ((x * x).sum(1) / d + EPS).rsqrt()
        y = torch.addcmul(x.new_zeros(d) if s["b"] is None else s["b"].double(), x * rstd[:, None], w)
        return (y, rstd) if case["rms"] else (y, mean, rstd)
    rstd, dy = s["rstd"].double()[:, None], s["dy"].double()
    if not case["rms"]:
        x = x - s["mean"].double()[:, None]
    x = x * rstd
    dw = torch.einsum("nd,nd->d", dy, x)
    db = torch.ones(n, dtype=torch.float64, device=x.device) @ dy
    dy *= w
    along = (dy * x).sum(1, keepdim=True) / d
    flat = 0.0 if case["rms"] else dy.sum(1, keepdim=True) / d
    dx = torch.addcmul(dy - flat, x, along, value=-1).mul_(rstd)
    return (dx, dw) if s["b"] is None else (dx, dw, db)


def _exact_grad(s):
    h, w = s["h"].double(), s["w"].double()
    n, real = h.shape[0], w.shape[0]
    x = torch.mm(h, w.T).to(torch.bfloat16).double()
    t, column = s["t"].double(), s["target"]
    inverse = torch.where(t > 0, 1 / t, 0.0)
    total = torch.zeros_like(x)
    picked = torch.zeros(n, dtype=torch.float64, device=x.device)
    if s["g_ref"] is not None:
        up = torch.where(t > 0, s["g_ref"].double() * inverse, 0.0)
        shift = torch.where(t > 0, s["lse"].double(), 0.0)
        total.addcmul_(torch.exp(x * inverse[:, None] - shift[:, None]), up[:, None], value=-1)
        picked += up * (1 - torch.exp(torch.where(t > 0, s["ref"].double(), 0.0)))
    if s["g_pol"] is not None:
        part, threshold = (s["state"][:, k].contiguous().view(torch.float32).double() for k in (0, 1))
        inside = (s["state"][:, 2] == 1) & (t > 0)
        up = torch.where(inside, s["g_pol"].double() * inverse, 0.0)
        shift = torch.where(inside, part, 0.0)
        weight = torch.exp(x * inverse[:, None] - shift[:, None]).masked_fill_(x < threshold[:, None], 0.0)
        weight[~inside] = 0.0
        total.addcmul_(weight, up[:, None], value=-1)
        picked += up * (1 - torch.exp(torch.where(inside, s["pol"].double(), 0.0)))
    total[torch.arange(n, device=x.device), column] = picked
    del x
    out = []
    if s["wants"] != "weight":
        out.append(torch.mm(total, w))
    if s["wants"] != "hidden":
        out.append(torch.mm(total.T, h))
    return out
