"""Measured cases of the serving operators: verification of drafted tokens
(draft_verify), microscaled 4-bit quantisation (mx4_quantize) and the LM-head
product with 4-bit operands (mx4_linear), with a plain form of each.

Verification. A batch of sequences, sequence s with K_s drafted tokens and
K_s + 1 rows of target logits. Both sides' per-row statistics (logprobs, the
records of the top-p support) are inputs, as the forward calls left them. Token
k is accepted when its random number lies below p/q; at the first that is not,
one token is drawn from max(p - q, 0), and from the last row's p where all are.

Microscaling. Blocks of 32 values along d share a power of two; a value is one
of +-{0, 0.5, 1, 1.5, 2, 3, 4, 6} times it. The product multiplies hidden
states, quantised on the way, with a projection that was quantised before.
"""
import math

import torch

own = False

HEAD_REAL, HEAD_PADDED, HEAD_D = 151936, 152576, 4096  # the benchmark's vocabulary and hidden width


def listed():
    head = dict(vocab_real=HEAD_REAL, vocab_padded=HEAD_PADDED)
    return [
        # one sequence, four drafted tokens, the whole vocabulary: an interactive user's step
        dict(name="verify 1 x 4", op="verify", n_seq=1, max_draft=4, ragged=False, top_p=1.0, temperature=1.0, draft="sampled", noise=0.5, **head),
        # a serving batch: ragged drafts (none, for some), nucleus support
        dict(name="verify 64 x 0..6 top-p", op="verify", n_seq=64, max_draft=6, ragged=True, top_p=0.95, temperature=0.7, draft="sampled", noise=0.5, **head),
        # no drafts: the sampler of a rollout batch, temperatures per request, greedy ones among them
        dict(name="sample 256", op="verify", n_seq=256, max_draft=0, ragged=False, top_p=1.0, temperature=-1.0, draft="sampled", noise=0.5, **head),
        # a large rollout batch on the whole vocabulary
        dict(name="verify 1024 x 3", op="verify", n_seq=1024, max_draft=3, ragged=False, top_p=1.0, temperature=1.0, draft="sampled", noise=0.5, **head),
        # a small adapter's matrix: latency
        dict(name="quantise 64 x 256", op="quantise", rows=64, d=256, pad=0),
        # an odd row count out of a wider buffer
        dict(name="quantise 4999 x 2080 strided", op="quantise", rows=4999, d=2080, pad=96),
        # the whole vocabulary projection, once a weight update
        dict(name="quantise 151936 x 4096", op="quantise", rows=HEAD_REAL, d=HEAD_D, pad=0),
        # one decoded token
        dict(name="linear 1", op="linear", rows=1, d=HEAD_D, **head),
        # a serving batch's rows, drafts with it
        dict(name="linear 48", op="linear", rows=48, d=HEAD_D, **head),
        # odd sizes throughout
        dict(name="linear 77 x 1056 x 50021", op="linear", rows=77, d=1056, vocab_real=50021, vocab_padded=50048),
        # a large batch with drafts
        dict(name="linear 640", op="linear", rows=640, d=HEAD_D, **head),
        # a validation's 8192 tokens
        dict(name="linear 8192", op="linear", rows=8192, d=HEAD_D, **head),
    ]


def _between(rng, lo, hi):
    """A whole number in [lo, hi], spread over its logarithm."""
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["verify", "verify", "quantise", "linear", "linear"])
    if op == "quantise":
        d = 32 * _between(rng, 1, 256)
        return dict(op=op, rows=_between(rng, 1, min(HEAD_REAL, HEAD_REAL * HEAD_D // d)), d=d, pad=rng.choice([0, 0, 8, 96]))
    if rng.random() < 0.4:
        real, padded = HEAD_REAL, HEAD_PADDED
    else:
        real = _between(rng, 300, HEAD_REAL)
        padded = (real + 63) // 64 * 64 + 64 * rng.choice([0, 0, 1, 5])
    if op == "linear":
        return dict(op=op, rows=_between(rng, 1, 4096), d=32 * _between(rng, 2, HEAD_D // 32), vocab_real=real, vocab_padded=padded)
    most = rng.choice([0, 1, 3, 5, 8])
    return dict(op=op, n_seq=_between(rng, 1, 384), max_draft=most, ragged=rng.random() < 0.5, top_p=rng.choice([1.0, 0.95, 0.99, 0.5]),
                temperature=rng.choice([1.0, 0.7, 1.3, -1.0]), draft=rng.choice(["sampled", "sampled", "token"]),
                noise=rng.choice([0.25, 0.5, 1.0]), vocab_real=real, vocab_padded=padded)


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------

def _rows_of_logits(gen, n, real, padded, dev):
    """BF16 logits N(0, 2.5^2) with one column of each row raised by 8; the pad columns hold -inf."""
    x = torch.full((n, padded), -math.inf, dtype=torch.bfloat16, device=dev)
    for at in range(0, n, 256):
        y = torch.randn((min(256, n - at), real), generator=gen, device=dev) * 2.5
        top = torch.randint(0, real, (y.shape[0], 1), generator=gen, device=dev)
        y.scatter_add_(1, top, torch.full_like(top, 8, dtype=y.dtype))
        x[at:at + 256, :real] = y.to(torch.bfloat16)
    return x


def _statistics(x, t, top_p, real, token):
    """What the forward call leaves of each row of `x`: (reference and policy logprob of `token`, lse, support records)."""
    n, dev = x.shape[0], x.device
    ref, pol, lse = (torch.empty(n, dtype=torch.float32, device=dev) for _ in range(3))
    state = torch.zeros((n, 4), dtype=torch.int32, device=dev)
    for at in range(0, n, 64):
        v = x[at:at + 64, :real].double()
        tt, tok = t[at:at + 64, None].double(), token[at:at + 64, None]
        greedy = tt == 0
        z = (v / torch.where(greedy, 1.0, tt)).float().double()
        full = torch.logsumexp(z, 1, keepdim=True)
        threshold = torch.full_like(full, -math.inf)
        if top_p < 1:
            order = torch.sort(z, 1, descending=True).values
            mass = torch.cumsum(torch.exp(order - full), 1)
            last = (mass < torch.tensor(top_p, dtype=torch.float32).item() * mass[:, -1:]).sum(1, keepdim=True).clamp(max=real - 1)
            kept = z >= torch.gather(order, 1, last)
            threshold = torch.where(kept, v, math.inf).amin(1, keepdim=True)
        inside = v >= threshold
        part = torch.logsumexp(torch.where(inside, z, -math.inf), 1, keepdim=True)
        zt, best = torch.gather(z, 1, tok), torch.argmax(v, 1, keepdim=True)
        point = torch.where(best == tok, 0.0, -math.inf).double()
        hit = torch.where(greedy, best == tok, torch.gather(inside, 1, tok))
        here = slice(at, at + v.shape[0])
        ref[here] = torch.where(greedy, point, zt - full)[:, 0].float()
        pol[here] = torch.where(greedy, point, torch.where(hit, zt - part, -math.inf))[:, 0].float()
        lse[here] = torch.where(greedy, math.nan, full)[:, 0].float()
        state[here, 0] = torch.where(greedy, math.nan, part)[:, 0].float().view(torch.int32)
        state[here, 1] = torch.where(greedy, -math.inf, threshold)[:, 0].float().view(torch.int32)
        state[here, 2] = hit[:, 0].int()
    return ref, pol, lse, state


def _drawn(gen, x, t, top_p, real):
    """A token of each row of `x`, drawn from its support by Gumbel maxima (the maximum itself in greedy rows)."""
    n, dev = x.shape[0], x.device
    tok = torch.zeros(n, dtype=torch.int64, device=dev)
    state = _statistics(x, t, top_p, real, tok)[3]
    for at in range(0, n, 64):
        v = x[at:at + 64, :real].float()
        tt, threshold = t[at:at + 64, None], state[at:at + 64, 1:2].view(torch.float32)
        noise = -torch.log(-torch.log(torch.rand(v.shape, generator=gen, device=dev).clamp(1e-10, 1 - 6e-8)))
        y = torch.where(tt == 0, v, v / torch.where(tt == 0, 1.0, tt) + noise)
        tok[at:at + 64] = torch.argmax(torch.where(v >= threshold, y, -math.inf), 1)
    return tok


def _prepare_verify(c, gen, dev):
    n, most, real, padded = c["n_seq"], c["max_draft"], c["vocab_real"], c["vocab_padded"]
    if c["ragged"]:  # every length from none to the most, in an order of the seed's
        count = (torch.arange(n, device=dev) % (most + 1))[torch.randperm(n, generator=gen, device=dev)]
    else:
        count = torch.full((n,), most, dtype=torch.int64, device=dev)
    start = torch.zeros(n + 1, dtype=torch.int64, device=dev)
    start[1:] = torch.cumsum(count, 0)
    n_draft = int(start[-1])
    if c["temperature"] < 0:  # per request, greedy ones among them
        t_seq = torch.tensor([0.7, 1.0, 1.3, 0.0], device=dev)[torch.randint(0, 4, (n,), generator=gen, device=dev)]
    else:
        t_seq = torch.full((n,), c["temperature"], device=dev)
    target = _rows_of_logits(gen, n_draft + n, real, padded, dev)
    seq = torch.repeat_interleave(torch.arange(n, device=dev), count)
    row = torch.arange(n_draft, device=dev) + seq
    t_row = torch.repeat_interleave(t_seq, count + 1).contiguous()
    t_draft = t_seq[seq].contiguous()
    draft = torch.full((n_draft, padded), -math.inf, dtype=torch.bfloat16, device=dev)
    for at in range(0, n_draft, 256):  # the drafter's logits: the target's with an error
        x = target[row[at:at + 256], :real].float()
        draft[at:at + 256, :real] = (x + c["noise"] * torch.randn(x.shape, generator=gen, device=dev)).to(torch.bfloat16)
    token = _drawn(gen, draft, t_draft, c["top_p"], real)
    scored = torch.zeros(n_draft + n, dtype=torch.int64, device=dev)
    scored[row] = token
    ref, pol, lse, state = _statistics(target, t_row, c["top_p"], real, scored)
    s = dict(op="verify", real=real, padded=padded, start=start, token=token, logits=target, temperature=t_row, ref=ref, pol=pol, lse=lse, state=state,
             accept_u=torch.rand(n_draft, generator=gen, device=dev, dtype=torch.float64),
             sample_u=torch.rand(n, generator=gen, device=dev, dtype=torch.float64), draft=None)
    if c["draft"] == "sampled" and n_draft:
        dpol, dstate = _statistics(draft, t_draft, c["top_p"], real, token)[1::2]
        s.update(draft=draft, draft_temperature=t_draft, draft_pol=dpol, draft_state=dstate)
    rows = n_draft + n
    s["out"] = dict(token_out=torch.empty(rows, dtype=torch.int64, device=dev), accepted_out=torch.empty(n, dtype=torch.int32, device=dev),
                    policy_out=torch.empty(rows, device=dev), ref_out=torch.empty(rows, device=dev))
    return s


def _prepare_quantise(c, gen, dev):
    x = torch.randn((c["rows"], c["d"] + c["pad"]), generator=gen, device=dev, dtype=torch.bfloat16)
    x *= 2.5 / 64
    # rows of unlike magnitude, as trained projections have
    x *= torch.exp2(torch.randint(-3, 4, (c["rows"], 1), generator=gen, device=dev)).to(torch.bfloat16)
    return dict(op="quantise", x=x[:, :c["d"]])


def _prepare_linear(c, gen, dev):
    n, d, real = c["rows"], c["d"], c["vocab_real"]
    hidden = torch.randn((n, d), generator=gen, device=dev).to(torch.bfloat16)
    codes, scales = [], []
    for at in range(0, real, 16384):
        w = torch.randn((min(16384, real - at), d), generator=gen, device=dev) * (2.5 / math.sqrt(d))
        a, b = _codes(w.to(torch.bfloat16))
        codes.append(a)
        scales.append(b)
    codes, scales = torch.cat(codes), torch.cat(scales)
    return dict(op="linear", real=real, padded=c["vocab_padded"], hidden=hidden, codes=codes, scales=scales, packed=_packed(codes, scales),
                out=torch.empty((n, c["vocab_padded"]), dtype=torch.bfloat16, device=dev))


def _packed(codes, scales):
    """The projection in the layout that the product reads, as a program keeps it: 32 rows x 64 values a KiB, lane by lane
    (codes [rows/32][d/64][2][32][16], scales [rows/32][d/256][2][32][4]); rows and values that are missing are zeros."""
    n, b = scales.shape
    rows, wide = -(-n // 32) * 32, -(-b // 8) * 8
    c = torch.zeros((rows, wide, 16), dtype=torch.uint8, device=codes.device)
    c[:n, :b] = codes.view(n, b, 16)
    s = torch.zeros((rows, wide), dtype=torch.uint8, device=codes.device)
    s[:n, :b] = scales
    c = c.view(rows // 32, 32, wide // 2, 2, 16).permute(0, 2, 3, 1, 4).contiguous().view(-1)
    s = s.view(rows // 32, 32, wide // 8, 4, 2).permute(0, 2, 4, 1, 3).contiguous().view(-1)
    return c, s


def prepare(case, seed):
    dev = torch.device("cuda", torch.cuda.current_device())
    gen = torch.Generator(device=dev)
    gen.manual_seed(seed)
    return {"verify": _prepare_verify, "quantise": _prepare_quantise, "linear": _prepare_linear}[case["op"]](case, gen, dev)


# ---------------------------------------------------------------------------
# the operators
# ---------------------------------------------------------------------------

def run(state):
    return {"verify": _verify, "quantise": _quantise, "linear": _linear}[state["op"]](state)


def _verify(s):
    if own:
        import invariant_token_log_fp32_amd as rlk
        more = {}
        if s["draft"] is not None:
            more = dict(draft_logits=s["draft"], draft_temperature=s["draft_temperature"], draft_policy_logp=s["draft_pol"],
                        draft_support_state=s["draft_state"])
        token, accepted, policy, ref = rlk.draft_verify(
            s["logits"], s["token"], s["start"], s["accept_u"], s["sample_u"], temperature=s["temperature"], policy_logp=s["pol"],
            ref_logp=s["ref"], lse=s["lse"], support_state=s["state"], vocab_real=s["real"], vocab_padded=s["padded"], **s["out"], **more)
        return dict(token=token, accepted=accepted, policy=policy, ref=ref)
    real, start, token, n_draft, n_rows = s["real"], s["start"], s["token"], s["token"].shape[0], s["logits"].shape[0]
    n = start.shape[0] - 1
    dev = start.device
    count = start[1:] - start[:-1]
    seq = torch.repeat_interleave(torch.arange(n, device=dev), count, output_size=n_draft)
    place = torch.arange(n_draft, device=dev)
    row = place + seq
    # which drafted tokens stay: up to the first whose number is not below p / q
    lp = s["pol"][row].double()
    lq = s["draft_pol"].double() if s["draft"] is not None else torch.zeros_like(lp)
    if s["draft"] is not None:
        lq = torch.where(s["draft_temperature"] == 0, 0.0, lq)
    stays = s["accept_u"] < torch.exp(lp - lq)
    stop = count.clone()
    stop.scatter_reduce_(0, seq, torch.where(stays, count[seq], place - start[seq]), "amin")
    # the distribution that the last token comes from
    at = start[:-1] + torch.arange(n, device=dev) + stop
    rejected = (stop < count)[:, None]
    drawn_at = torch.clamp(start[:-1] + stop, max=max(0, n_draft - 1))

    def probabilities(logits, temperature, records, rows):
        x, t = logits[rows, :real].double(), temperature[rows, None].double()
        part, threshold = records[rows, 0:1].view(torch.float32).double(), records[rows, 1:2].view(torch.float32).double()
        z = (x / torch.where(t == 0, 1.0, t)).float().double()
        p = torch.where(x >= threshold, torch.exp(z - part), 0.0)
        point = torch.arange(real, device=dev) == torch.argmax(x, 1, keepdim=True)
        return torch.where(t == 0, point.double(), p), z, part

    p, z, part = probabilities(s["logits"], s["temperature"], s["state"], at)
    r = p
    if n_draft:
        chosen = token[drawn_at][:, None]
        point = (torch.arange(real, device=dev) == chosen).double()
        if s["draft"] is not None:
            q = probabilities(s["draft"], s["draft_temperature"], s["draft_state"], drawn_at)[0]
            q = torch.where(s["draft_temperature"][drawn_at, None] == 0, point, q)
        else:
            q = point
        r = torch.where(rejected, torch.clamp(p - q, min=0.0), p)
    below = torch.cumsum(r, 1)
    pick = (below <= s["sample_u"][:, None] * below[:, -1:]).sum(1)
    last = torch.where(r > 0, torch.arange(real, device=dev), 0).amax(1)
    pick = torch.minimum(pick, last)
    if n_draft:  # p is nowhere above q: the drafted token itself
        pick = torch.where((below[:, -1] == 0), chosen[:, 0], pick)
    greedy = s["temperature"][at] == 0
    zt = torch.gather(z, 1, pick[:, None])[:, 0]
    new_policy = torch.where(greedy, 0.0, zt - part[:, 0]).float()
    new_ref = torch.where(greedy, 0.0, zt - s["lse"][at].double()).float()
    # the tokens that come out, in the rows' places
    out = torch.full((n_rows,), -1, dtype=torch.int64, device=dev)
    policy, ref = torch.zeros(n_rows, device=dev), torch.zeros(n_rows, device=dev)
    kept = place - start[seq] < stop[seq]
    out[row] = torch.where(kept, token, -1)
    policy[row] = torch.where(kept, s["pol"][row], 0.0)
    ref[row] = torch.where(kept, s["ref"][row], 0.0)
    out[at], policy[at], ref[at] = pick, new_policy, new_ref
    return dict(token=out, accepted=stop.int(), policy=policy, ref=ref)


def _scale_exponents(x):
    """The shared exponents of blocks of 32 values: floor(log2 of the largest magnitude) - 2."""
    most = x.abs().amax(-1)
    return torch.where(most > 0, torch.frexp(most).exponent - 3, -127).clamp(-127, 127)


def _codes(x):
    """The 4-bit codes (two a byte, the even value low) and the scale bytes of rows of BF16 values."""
    x = x.float().view(x.shape[0], -1, 32)
    e = _scale_exponents(x)
    y = torch.ldexp(x.abs(), -e[..., None])
    # nearest of 0, 0.5, 1, 1.5, 2, 3, 4, 6, ties to the even code
    code = ((y > 0.25).byte() + (y >= 0.75).byte() + (y > 1.25).byte() + (y >= 1.75).byte() + (y > 2.5).byte() + (y >= 3.5).byte()
            + (y > 5).byte() + 8 * torch.signbit(x).byte())
    return (code[..., 0::2] | (code[..., 1::2] << 4)).view(x.shape[0], -1), (e + 127).byte()


def _values(codes, scales):
    """What codes and scale bytes stand for, in 32 bits."""
    levels = torch.tensor([0, 0.5, 1, 1.5, 2, 3, 4, 6, -0.0, -0.5, -1, -1.5, -2, -3, -4, -6], device=codes.device)
    both = torch.stack((codes & 15, codes >> 4), -1).view(codes.shape[0], -1, 32).int()
    return torch.ldexp(levels[both], (scales.int() - 127)[..., None]).view(codes.shape[0], -1)


def _quantise(s):
    if own:
        import invariant_token_log_fp32_amd as rlk
        return dict(values=rlk.mx4_quantize(s["x"], return_values=True)[2])
    return dict(values=_values(*_codes(s["x"])).to(torch.bfloat16))


def _linear(s):
    if own:
        import invariant_token_log_fp32_amd as rlk
        return dict(logits=rlk.mx4_linear(s["hidden"], *s["packed"], vocab_real=s["real"], vocab_padded=s["padded"], out=s["out"]))
    h = _values(*_codes(s["hidden"]))
    x = torch.full((h.shape[0], s["padded"]), -math.inf, dtype=torch.bfloat16, device=h.device)
    x[:, :s["real"]] = (h @ _values(s["codes"], s["scales"]).t()).to(torch.bfloat16)
    return dict(logits=x)


def work(case):
    if case["op"] == "quantise":
        n = case["rows"] * case["d"]
        # the BF16 values in; codes, scales and the values they stand for out
        return dict(bytes=n * (2 + 17 / 32 + 2), flops=n)
    if case["op"] == "linear":
        n, d, real = case["rows"], case["d"], case["vocab_real"]
        return dict(bytes=2 * n * d + real * d * 17 / 32 + 2 * n * case["vocab_padded"], flops=2 * n * d * real)
    # the row of target logits that the last token comes from and, where a drafted token is refused, the draft's row:
    # about one token in five is, at the listed cases' noise
    mean = case["max_draft"] / 2 if case["ragged"] else case["max_draft"]
    rows = case["n_seq"] * (1 + (1 - 0.8 ** mean if case["draft"] == "sampled" else 0))
    tokens = case["n_seq"] * (2 * mean + 1)
    return dict(bytes=2 * rows * case["vocab_real"] + 80 * tokens, flops=4 * rows * case["vocab_real"])


# ---------------------------------------------------------------------------
# the definitions in 64 bits
# ---------------------------------------------------------------------------

def exact(case, seed):
    s = prepare(case, seed)
    return {"verify": _exact_verify, "quantise": _exact_quantise, "linear": _exact_linear}[case["op"]](s)


def _distribution(logits, t, part, threshold, real):
    x = logits[:real].double()
    if t == 0:
        p = torch.zeros_like(x)
        p[int((x == x.max()).nonzero()[0])] = 1
        return p
    z = (logits[:real].float() / torch.full_like(logits[:real].float(), t)).double()
    return torch.exp(z - part) * (x >= threshold)


def _exact_verify(s):
    start, real = s["start"].tolist(), s["real"]
    tokens, u, v = s["token"].tolist(), s["accept_u"].tolist(), s["sample_u"].tolist()
    pol, ref, lse, t = s["pol"].tolist(), s["ref"].tolist(), s["lse"].tolist(), s["temperature"].tolist()
    record = s["state"][:, :2].contiguous().view(torch.float32).tolist()
    n = len(start) - 1
    rows = s["logits"].shape[0]
    out, accepted = [-1] * rows, [0] * n
    policy, reference = [0.0] * rows, [0.0] * rows
    if s["draft"] is not None:
        dpol, dt, drecord = s["draft_pol"].tolist(), s["draft_temperature"].tolist(), s["draft_state"][:, :2].contiguous().view(torch.float32).tolist()
    for i in range(n):
        k, base = 0, start[i] + i
        count = start[i + 1] - start[i]
        while k < count:
            j = start[i] + k
            lq = dpol[j] if s["draft"] is not None and dt[j] != 0 else 0.0
            if not u[j] < math.exp(min(700.0, pol[base + k] - lq)):
                break
            out[base + k], policy[base + k], reference[base + k] = tokens[j], pol[base + k], ref[base + k]
            k += 1
        accepted[i] = k
        at, j = base + k, start[i] + k
        r = _distribution(s["logits"][at], t[at], *record[at], real)
        if k < count:
            if s["draft"] is not None and dt[j] != 0:
                r = (r - _distribution(s["draft"][j], dt[j], *drecord[j], real)).clamp(min=0)
            else:
                r = r.clone()
                r[tokens[j]] = max(0.0, float(r[tokens[j]]) - 1)
        sums = torch.cumsum(r, 0)
        over = (sums > v[i] * sums[-1]).nonzero()
        pick = int(over[0]) if len(over) else tokens[j]
        out[at] = pick
        if t[at] != 0:
            z = float(s["logits"][at, pick].float() / torch.tensor(t[at], dtype=torch.float32, device=sums.device))
            policy[at], reference[at] = z - record[at][0], z - lse[at]
    f = lambda a: torch.tensor(a, dtype=torch.float64)  # noqa: E731
    return dict(token=torch.tensor(out), accepted=torch.tensor(accepted, dtype=torch.int32), policy=f(policy), ref=f(reference))


_GRID = [0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0]


def _exact_values(x):
    """Blocks of 32 in 64 bits: the grid's nearest value to |x| / 2^e, the one with the even place on a tie."""
    out = torch.empty(x.shape, dtype=torch.float64, device=x.device)
    for at in range(0, x.shape[0], 8192):
        v = x[at:at + 8192].double().unflatten(1, (-1, 32))
        top = v.abs().amax(-1, keepdim=True)
        e = torch.floor(torch.log2(torch.where(top > 0, top, 1.0))) - 2
        y = v.abs() / torch.exp2(e)
        best, off = torch.zeros_like(y), y.clone()
        for place in (2, 4, 6, 1, 3, 5, 7):  # even places first: an odd one has to be nearer
            away = (y - _GRID[place]).abs()
            nearer = away < off
            best = torch.where(nearer, _GRID[place], best)
            off = torch.where(nearer, away, off)
        out[at:at + 8192] = (torch.sign(v) * best * torch.exp2(e)).flatten(1)
    return out


def _exact_quantise(s):
    return dict(values=_exact_values(s["x"]))


def _exact_linear(s):
    h = _exact_values(s["hidden"])
    x = torch.full((h.shape[0], s["padded"]), -math.inf, dtype=torch.float64, device=h.device)
    grid = torch.tensor(_GRID + [-g for g in _GRID], dtype=torch.float64, device=h.device)
    for at in range(0, s["real"], 16384):
        codes, scales = s["codes"][at:at + 16384].long(), s["scales"][at:at + 16384]
        w = torch.empty((codes.shape[0], 2 * codes.shape[1]), dtype=torch.float64, device=h.device)
        w[:, 0::2], w[:, 1::2] = grid[codes % 16], grid[codes // 16]
        w *= torch.exp2(scales.double() - 127).repeat_interleave(32, 1)
        x[:, at:at + codes.shape[0]] = h @ w.t()
    return dict(logits=x)
