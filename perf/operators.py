"""The token-loss operators as they are measured: log probabilities of given
tokens (with entropy and the top alternatives) and distillation from a
teacher's top logits, each as the forward pass alone, the backward pass from
the forward's statistics, and both in one call.

``own`` false: ``run`` computes them in elementary torch operations, in 32 bits,
rounded once at the end.  ``own`` true: ``run`` calls the library's entry points.

Vocabularies are those of the repository's workloads (50304 of the GPT-2
Large-sized model, 128256 of the 8B Llama-shaped one), 50257 columns kept in
rows of 50304 or back to back, and generic odd ones; rows are the tokens of a
batch (1024 is the GPT-2 Large context).
"""
import math

import torch

own = False

RENORM, TAIL = "renorm", "tail"
PAD_EVERY = 8        # with "padding", every eighth row is a padding row
MASK_KEEP = 16       # with "masked", one token in sixteen stays allowed


def _case(name, op, form, rows, vocab, dtype, **more):
    c = {"name": name, "op": op, "form": form, "rows": rows, "vocab": vocab, "stride": vocab,
         "dtype": dtype, "scale": 1.0, "top": 0, "entropy": False, "padding": False,
         "masked": False, "mode": ""}
    c.update(more)
    return c


def listed():
    return [
        # one sampled token's record while serving: its log probability, the
        # entropy and five alternatives
        _case("score-1x50304-top5", "logprob", "forward", 1, 50304, "bf16", top=5, entropy=True),
        # a decoding batch under a grammar mask (-inf outside it), twenty alternatives
        _case("score-64x128256-top20", "logprob", "forward", 64, 128256, "bf16", top=20,
              entropy=True, masked=True, scale=1.25),
        # scoring a batch of sampled sequences for policy training
        _case("score-4096x128256", "logprob", "forward", 4096, 128256, "bf16", entropy=True),
        # a teacher's record for distillation: the 64 top tokens of every position
        _case("record-2048x128256-top64", "logprob", "forward", 2048, 128256, "bf16", top=64),
        # a policy gradient's backward pass with an entropy bonus, fp32 logits
        _case("policy-backward-2048x50304", "logprob", "backward", 2048, 50304, "f32", entropy=True),
        # the language-model loss and its gradient: one GPT-2 Large context ...
        _case("lm-1024x50304", "logprob", "fused", 1024, 50304, "bf16", padding=True),
        # ... and the largest, a batch of the 8B model
        _case("lm-8192x128256", "logprob", "fused", 8192, 128256, "bf16"),
        # an odd vocabulary in padded rows, fp32, padding tokens in the batch
        _case("lm-777x50257-f32", "logprob", "fused", 777, 50257, "f32", stride=50304, padding=True),
        # one short sequence evaluated against its teacher
        _case("distill-3x50257", "distill", "forward", 3, 50257, "f32", top=8, mode=RENORM),
        # a distillation batch: loss and gradient, the rest of the vocabulary as one bucket
        _case("distill-4096x128256", "distill", "fused", 4096, 128256, "bf16", top=64, mode=TAIL),
        # odd rows back to back, renormalised over a hundred tokens, at a temperature
        _case("distill-511x50257", "distill", "fused", 511, 50257, "bf16", top=100, mode=RENORM,
              scale=0.5, padding=True),
        # the backward pass alone, as an autograd graph calls it
        _case("distill-backward-2048x128256", "distill", "backward", 2048, 128256, "bf16", top=32,
              mode=TAIL),
    ]


def draw(rng):
    op = rng.choice(["logprob", "distill"])
    form = rng.choice(["forward", "backward", "fused"])
    vocab = int(round(math.exp(rng.uniform(math.log(1000), math.log(131072)))))
    # not above the largest listed case's elements
    most = min(8192, 8192 * 128256 // (2 * vocab))
    rows = int(round(math.exp(rng.uniform(0.0, math.log(most)))))
    stride = vocab if rng.random() < 0.5 else vocab + rng.randrange(1, 64)
    c = _case("", op, form, rows, vocab, rng.choice(["bf16", "f32"]), stride=stride,
              scale=rng.choice([1.0, 0.5, 0.8, 1.25, 2.0]), padding=rng.random() < 0.3)
    if op == "logprob":
        c["entropy"] = rng.random() < 0.5
        if form == "forward":
            c["top"] = rng.choice([0, 1, 5, 20, 64, 200])
            c["masked"] = rng.random() < 0.3 and vocab >= 16000
    else:
        c["top"] = rng.choice([1, 8, 32, 64, 100, 256])
        c["mode"] = rng.choice([RENORM, TAIL])
    del c["name"]
    return c


# -- inputs -------------------------------------------------------------------

def _dtype(case):
    return torch.bfloat16 if case["dtype"] == "bf16" else torch.float32


def _padding_rows(case):
    return case["rows"] // PAD_EVERY if case["padding"] else 0


def _blocks(rows, vocab):
    """Row ranges of about 2^28 elements, which bound the intermediates."""
    n = max(1, min(rows, (1 << 28) // max(vocab, 1)))
    return [(a, min(a + n, rows)) for a in range(0, rows, n)]


def prepare(case, seed):
    dev = torch.device("cuda")
    gen = torch.Generator(device=dev).manual_seed(seed)
    R, V, K = case["rows"], case["vocab"], case["top"]
    st = {"case": case}
    buf = torch.empty(R, case["stride"], dtype=_dtype(case), device=dev)
    st["logits"] = logits = buf[:, :V]
    tokens = torch.randint(0, V, (R,), generator=gen, device=dev)
    pad = None
    if case["padding"]:
        pad = torch.arange(R, device=dev) % PAD_EVERY == PAD_EVERY - 1
    if case["op"] == "distill":
        st["top_index"] = torch.empty(R, K, dtype=torch.int32, device=dev)
        st["top_value"] = torch.empty(R, K, device=dev)
    for a, b in _blocks(R, V):
        # a trained model's rows: spread logits, most given tokens likely
        x = torch.randn(b - a, V, generator=gen, device=dev) * 2.5 - 4.0
        t = tokens[a:b, None]
        x.scatter_add_(1, t, torch.rand(b - a, 1, generator=gen, device=dev) * 14.0)
        if case["masked"]:
            keep = torch.rand(b - a, V, generator=gen, device=dev) < 1.0 / MASK_KEEP
            keep.scatter_(1, t, True)
            x.masked_fill_(~keep, -math.inf)
        buf[a:b].zero_()
        logits[a:b].copy_(x)
        if case["op"] == "distill":
            y = x + torch.randn(b - a, V, generator=gen, device=dev)
            y = torch.log_softmax(y * case["scale"], dim=1)
            v, i = torch.topk(y, K, dim=1)
            st["top_index"][a:b], st["top_value"][a:b] = i.to(torch.int32), v
    if pad is not None:
        tokens[pad] = -1
        if case["op"] == "distill":
            st["top_index"][pad] = -1
    st["tokens"] = tokens
    n = max(1, R - _padding_rows(case))
    up = (0.5 + torch.rand(R, generator=gen, device=dev)) / n
    if case["op"] == "logprob":
        st["d_logprob"] = -up
        st["d_entropy"] = torch.full((R,), -0.01 / n, device=dev) if case["entropy"] else None
    else:
        st["d_loss"] = up
    if case["form"] == "backward":
        _forward_statistics(st)
    if own:
        import fsdp_sharded_optimizer_flat_amd as z
        st["workspace"] = torch.empty(z.zero_loss_workspace_bytes(R, V, K), dtype=torch.uint8,
                                      device=dev)
        st["out"] = _outputs(case, dev)
    return st


def _forward_statistics(st):
    """What the forward pass has left for the backward one: each row's largest
    logit and the logarithm of its sum of exponentials relative to it (for
    distillation also over the tokens the teacher does not list), the entropy."""
    case, s = st["case"], st["case"]["scale"]
    R, V = case["rows"], case["vocab"]
    width = 2 if case["op"] == "logprob" else 4
    stats = torch.zeros(R, width, device="cuda")
    ent = torch.zeros(R, device="cuda")
    for a, b in _blocks(R, 2 * V):
        x = st["logits"][a:b].double()

        def max_and_log_sum(x):
            m = x.amax(1)
            return m, torch.exp((x - m[:, None]) * s).sum(1).log()

        m, ls = max_and_log_sum(x)
        stats[a:b, 0], stats[a:b, 1] = m, ls
        if width == 2:
            lp = (x - m[:, None]) * s - ls[:, None]
            ent[a:b] = -(lp.exp() * lp).sum(1)
        else:
            x.scatter_(1, st["top_index"][a:b].long().clamp(min=0), -math.inf)
            m, ls = max_and_log_sum(x)
            stats[a:b, 2], stats[a:b, 3] = m, ls
    st["stats"], st["row_entropy"] = stats, ent


def _outputs(case, dev):
    R, V, K = case["rows"], case["vocab"], case["top"]
    f = lambda *s: torch.empty(*s, device=dev)
    o = {}
    if case["op"] == "logprob" and case["form"] != "backward":
        o["logprob"] = f(R)
        o["entropy"] = f(R) if case["entropy"] else None
        if K:
            o["top_index"] = torch.empty(R, K, dtype=torch.int32, device=dev)
            o["top_logprob"] = f(R, K)
    if case["op"] == "distill" and case["form"] != "backward":
        o["loss"] = f(R)
    if case["form"] != "forward":
        o["d_logits"] = torch.empty(R, V, dtype=_dtype(case), device=dev)
    return o


# -- one pass --------------------------------------------------------------------

def run(st):
    return _run_own(st) if own else _run_plain(st)


def _run_own(st):
    import fsdp_sharded_optimizer_flat_amd as z
    case, o = st["case"], st["out"]
    x, s, form = st["logits"], case["scale"], case["form"]
    if case["op"] == "logprob":
        if form == "forward":
            z.zero_logprob(x, st["tokens"], scale=s, logprob=o["logprob"], entropy=o["entropy"],
                           top_index=o.get("top_index"), top_logprob=o.get("top_logprob"),
                           workspace=st["workspace"])
        elif form == "backward":
            z.zero_logprob_grad(x, st["tokens"], st["stats"], o["d_logits"], scale=s,
                                d_logprob=st["d_logprob"], d_entropy=st["d_entropy"],
                                entropy=st["row_entropy"] if case["entropy"] else None)
        else:
            z.zero_logprob_fused(x, st["tokens"], o["d_logits"], scale=s, d_logprob=st["d_logprob"],
                                 d_entropy=st["d_entropy"], logprob=o["logprob"],
                                 entropy=o["entropy"], workspace=st["workspace"])
    else:
        mode = z.ZERO_DISTILL_TAIL if case["mode"] == TAIL else z.ZERO_DISTILL_RENORM
        if form == "forward":
            z.zero_distill(x, st["top_index"], st["top_value"], mode, scale=s, loss=o["loss"],
                           workspace=st["workspace"])
        elif form == "backward":
            z.zero_distill_grad(x, st["top_index"], st["top_value"], mode, st["stats"],
                                st["d_loss"], o["d_logits"], scale=s)
        else:
            z.zero_distill_fused(x, st["top_index"], st["top_value"], mode, st["d_loss"],
                                 o["d_logits"], scale=s, loss=o["loss"], workspace=st["workspace"])
    return o


def _run_plain(st):
    case = st["case"]
    if case["op"] == "logprob":
        return _plain_logprob(st)
    return _plain_distill(st)


def _plain_logprob(st):
    case = st["case"]
    x = st["logits"].float()
    t = st["tokens"]
    live = (t >= 0)[:, None]
    at = t.clamp(min=0)[:, None]
    if case["form"] == "backward":
        m, ls = st["stats"][:, :1], st["stats"][:, 1:]
    else:
        m = x.amax(1, keepdim=True)
        ls = torch.exp((x - m) * case["scale"]).sum(1, keepdim=True).log()
    logp = (x - m) * case["scale"] - ls
    o = {}
    ent = None
    if case["entropy"]:
        plogp = torch.where(logp > -math.inf, torch.exp(logp) * logp, 0.0)
        ent = -plogp.sum(1, keepdim=True)
    if case["form"] != "backward":
        o["logprob"] = torch.where(live, logp.gather(1, at), 0.0)[:, 0]
        o["entropy"] = torch.where(live, ent, 0.0)[:, 0] if ent is not None else None
    if case["top"]:
        # a whole number for each logit that grows with its value and falls
        # with its index, so that ties go to the lowest index
        bits = (x + 0.0).view(torch.int32).long()
        order = torch.where(bits >= 0, bits, -(bits & 0x7fffffff))
        key = order * (1 << 24) + ((1 << 24) - 1 - torch.arange(x.shape[1], device=x.device))
        i = torch.topk(key, case["top"], dim=1).indices
        lp = logp.gather(1, i)
        none = ~live | (lp == -math.inf)
        o["top_index"] = torch.where(none, -1, i).to(torch.int32)
        o["top_logprob"] = torch.where(none, -math.inf, lp)
    if case["form"] != "forward":
        p = torch.exp(logp)
        d = st["d_logprob"][:, None]
        g = -p * d
        g.scatter_add_(1, at, d)
        if case["entropy"]:
            g -= st["d_entropy"][:, None] * torch.where(p > 0, p * (logp + ent), 0.0)
        o["d_logits"] = torch.where(live, g * case["scale"], 0.0).to(_dtype(case))
    return o


def _plain_distill(st):
    case, s = st["case"], st["case"]["scale"]
    x = st["logits"].float()
    i = st["top_index"].long()
    valid = i >= 0
    live = valid.any(1, keepdim=True)
    at = i.clamp(min=0)
    val = torch.where(valid, st["top_value"].double(), -math.inf)
    if case["mode"] == RENORM:
        # the values are log probabilities at the temperature already
        e = torch.exp((val - val.amax(1, keepdim=True).clamp(min=-1e300)))
        q = e / e.sum(1, keepdim=True).clamp(min=1e-300)
        rest = torch.zeros_like(q[:, :1])
    else:
        q = torch.exp(val)
        rest = 1.0 - q.sum(1, keepdim=True)
        rest = torch.where(rest < 2.0 ** -20, 0.0, rest)
    total = (q.sum(1, keepdim=True) + rest).float()
    unlisted = x.scatter(1, at, -math.inf)
    if case["form"] == "backward":
        m, ls, mt, lst = st["stats"].split(1, 1)
    else:
        m = x.amax(1, keepdim=True)
        ls = torch.exp((x - m) * s).sum(1, keepdim=True).log()
        mt = unlisted.amax(1, keepdim=True)
        lst = torch.exp((unlisted - mt) * s).sum(1, keepdim=True).log()
    logp = ((x.gather(1, at) - m) * s - ls).double()
    log_rest = ((mt - m) * s + lst - ls).double()
    o = {}
    if case["form"] != "backward":
        kl = torch.where(q > 0, q * (q.log() - logp), 0.0).sum(1, keepdim=True)
        kl += torch.where(rest > 0, rest * (rest.log() - log_rest), 0.0)
        o["loss"] = torch.where(live, kl, 0.0)[:, 0].float()
    if case["form"] != "forward":
        w = st["d_loss"][:, None] * s
        share = torch.exp((unlisted - mt) * s - lst)       # of the unlisted tokens' probability
        g = share * (total * log_rest.exp().float() - rest.float()) * w
        g.scatter_(1, at, ((total * logp.exp() - q) * w).float())
        o["d_logits"] = torch.where(live, g, 0.0).to(_dtype(case))
    return o


# -- what a pass cannot do without ---------------------------------------------------

def work(case):
    R, V, K = case["rows"], case["vocab"], case["top"]
    es = 2 if case["dtype"] == "bf16" else 4
    live = R - _padding_rows(case)
    n = live * V
    byt, flops = float(n * es), 4.0 * n              # logits in; difference, scale, exp, sum
    if case["op"] == "logprob":
        byt += 8.0 * R                               # tokens
        if case["form"] != "backward":
            byt += 4.0 * R * (1 + case["entropy"]) + 8.0 * R * K
        flops += 2.0 * n * case["entropy"]
    else:
        byt += 8.0 * R * K + 4.0 * R                 # the teacher's record, the losses
    if case["form"] != "forward":
        byt += float(R * V * es) + 4.0 * R           # gradient out, the weight of each row
        flops += 2.0 * n + 2.0 * n * case["entropy"]
    if case["form"] == "backward":
        byt += 8.0 * R * (1 if case["op"] == "logprob" else 2) + 4.0 * R * case["entropy"]
        flops -= 1.0 * n                             # the sum is there already
    return {"bytes": byt, "flops": flops}


# -- the definition in 64 bits -----------------------------------------------------------

def exact(case, seed):
    global own
    kept, own = own, False
    try:
        st = prepare(case, seed)
    finally:
        own = kept
    R, V = case["rows"], case["vocab"]
    parts = [_exact_rows(st, a, b) for a, b in _blocks(R, 2 * V)]
    o = {}
    for k in parts[0]:
        o[k] = None if parts[0][k] is None else torch.cat([p[k] for p in parts])
    return o


def _exact_rows(st, a, b):
    case, s, f64 = st["case"], st["case"]["scale"], torch.float64
    z = st["logits"][a:b].to(f64) * s
    lp = z - torch.logsumexp(z, 1)[:, None]
    p = lp.exp()
    grad = case["form"] != "forward"
    out = {}
    if case["op"] == "logprob":
        tok = st["tokens"][a:b]
        on = tok >= 0
        hot = torch.zeros(p.shape, dtype=torch.bool, device=p.device)
        hot[on, tok[on]] = True
        ent = -torch.special.xlogy(p, p).sum(1) if case["entropy"] else None
        if case["form"] != "backward":
            out["logprob"] = lp.masked_fill(~hot, 0.0).sum(1)
            out["entropy"] = None if ent is None else ent * on
        if case["top"]:
            order = torch.sort(z, dim=1, descending=True, stable=True)[1][:, :case["top"]]
            v = torch.take_along_dim(lp, order, 1)
            gone = torch.isinf(v) | ~on[:, None]
            out["top_index"] = order.masked_fill(gone, -1).to(torch.int32)
            out["top_logprob"] = v.masked_fill(gone, -math.inf)
        if grad:
            g = (hot.to(f64) - p) * st["d_logprob"][a:b, None].to(f64)
            if case["entropy"]:
                g -= st["d_entropy"][a:b, None].to(f64) * (torch.special.xlogy(p, p) + p * ent[:, None])
            out["d_logits"] = g * on[:, None] * s
        return out
    idx, val = st["top_index"][a:b], st["top_value"][a:b].to(f64)
    on = (idx >= 0)[:, 0]                        # rows are listed whole or not at all here
    idx = torch.where(idx >= 0, idx, 0).long()
    q = torch.softmax(val, 1) if case["mode"] == RENORM else val.exp()
    tail = 1.0 - q.sum(1)
    tail = torch.where(tail >= 2.0 ** -20, tail, torch.zeros_like(tail))
    if case["mode"] == RENORM:
        tail = torch.zeros_like(tail)
    full_q = torch.zeros_like(p).scatter(1, idx, q)
    seen = torch.zeros_like(p, dtype=torch.bool).scatter(1, idx, True)
    log_tail = torch.logsumexp(lp.masked_fill(seen, -math.inf), 1)
    if case["form"] != "backward":
        loss = torch.special.xlogy(q, q).sum(1) - (q * lp.gather(1, idx)).sum(1)
        loss = loss + torch.special.xlogy(tail, tail) - tail * log_tail
        out["loss"] = loss * on
    if grad:
        sum_q = (q.sum(1) + tail)[:, None]
        within = torch.where(seen, 0.0, torch.exp(lp - log_tail[:, None]))
        g = sum_q * p - full_q - tail[:, None] * within
        out["d_logits"] = g * (st["d_loss"][a:b].to(f64) * s * on)[:, None]
    return out
