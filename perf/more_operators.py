"""The operators around the token losses as they are measured: what turns
tokens' log probabilities into a loss (the clipped policy loss with a KL term,
the preference loss over pairs), the embedding lookup that a forward pass starts
at with the gradient that a backward pass ends at, and the 8-bit activation
checkpoints in between with the weight gradient that is formed from them.

``own`` false: ``run`` computes them in elementary torch operations, in 32 bits
(the losses' per-token terms and sums in 64: ratios next to the clipping border,
differences of nearly equal log probabilities), rounded once at the end.
``own`` true: ``run`` calls the library's entry points.

Widths and vocabularies are those of the repository's workloads (hidden 1280,
50304 tokens of the GPT-2 Large-sized model; 4096, 14336, 128256 of the 8B
Llama-shaped one) and generic odd ones.
"""
import math

import torch

own = False

MEAN, SUM = "mean", "sum"
SIGMOID, HINGE, SQUARED = "sigmoid", "hinge", "squared"
BLOCK = 32           # elements of a checkpoint that share a scale


def listed():
    return [
        # one sampled answer's policy loss: where only latency counts
        _policy("policy-1x1024", 1, 1024, kl_coef=0.0, per_token=False, mode=MEAN),
        # a batch of 300 packed answers, an advantage and a KL term for every token
        _policy("policy-300x3400", 300, 1020001, kl_coef=0.05, per_token=True, mode=MEAN),
        # evaluating two preference pairs, forward only
        _preference("prefer-2x700", 2, 1399, gradient=False, kind=SIGMOID, mode=SUM),
        # a large batch of pairs with gradients, averaged over their lengths
        _preference("prefer-128x4000", 128, 1024000, gradient=True, kind=SIGMOID, mode=MEAN),
        # a decoding batch's rows
        _embed("embed-16x4096", 16, 4096, 128256, "bf16", "bf16", scale=1.0),
        # a training batch, scaled, odd rows of fp32 masters into bf16 activations
        _embed("embed-20001x1280", 20001, 1280, 50304, "f32", "bf16", scale=math.sqrt(1280.0)),
        # one GPT-2 Large context's gradient into its bucket
        _embed_grad("embed-grad-1024x1280", 1024, 1280, 50304, "bf16", "bf16"),
        # a batch of the 8B model: the whole table's gradient
        _embed_grad("embed-grad-16384x4096", 16384, 4096, 128256, "bf16", "bf16"),
        # one layer's checkpoint there and back: odd rows of fp32
        _pack("act8-777x1283", 777, 1283, "f32"),
        # the widest activation of an 8B model's batch
        _pack("act8-8192x14336", 8192, 14336, "bf16"),
        # a GPT-2 Large projection's gradient from one context, odd tokens, fp32 bucket
        _weight_grad("wgrad-1023x1280x1280", 1023, 1280, 1280, "f32"),
        # the 8B model's FFN
        _weight_grad("wgrad-8192x14336x4096", 8192, 14336, 4096, "bf16"),
    ]


def _policy(name, seqs, tokens, **more):
    c = {"name": name, "op": "policy", "seqs": seqs, "tokens": tokens, "gradient": True,
         "clip_low": 0.2, "clip_high": 0.28, "kl_coef": 0.05, "per_token": True, "mode": MEAN}
    c.update(more)
    return c


def _preference(name, pairs, tokens, **more):
    c = {"name": name, "op": "preference", "pairs": pairs, "tokens": tokens, "gradient": True,
         "kind": SIGMOID, "mode": SUM, "beta": 0.1, "margin": 0.0, "smoothing": 0.0,
         "reference": True}
    c.update(more)
    return c


def _embed(name, rows, hidden, vocab, dtype, out_dtype, scale):
    return {"name": name, "op": "embed", "rows": rows, "hidden": hidden, "vocab": vocab,
            "dtype": dtype, "out_dtype": out_dtype, "scale": scale}


def _embed_grad(name, rows, hidden, vocab, dtype, out_dtype, scale=1.0):
    return {"name": name, "op": "embed_grad", "rows": rows, "hidden": hidden, "vocab": vocab,
            "dtype": dtype, "out_dtype": out_dtype, "scale": scale}


def _pack(name, rows, cols, dtype):
    return {"name": name, "op": "act8", "rows": rows, "cols": cols, "dtype": dtype}


def _weight_grad(name, rows, out, cols, out_dtype):
    return {"name": name, "op": "wgrad", "rows": rows, "out": out, "cols": cols,
            "out_dtype": out_dtype}


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["policy", "preference", "embed", "embed_grad", "act8", "wgrad"])
    dtype, out = rng.choice(["bf16", "f32"]), rng.choice(["bf16", "f32"])
    if op in ("policy", "preference"):
        seqs = _log_int(rng, 1, 2048)
        tokens = min(1020000, seqs * _log_int(rng, 1, 8192) + rng.randrange(64))
        mode = rng.choice([MEAN, SUM])
        gradient = tokens > 8192 or rng.random() < 0.5       # small evaluations: forward only
        if op == "policy":
            c = _policy("", seqs, max(tokens, 1), clip_low=rng.choice([0.1, 0.2, 0.3]),
                        clip_high=rng.choice([0.2, 0.28, 1.0]), kl_coef=rng.choice([0.0, 0.01, 0.2]),
                        per_token=rng.random() < 0.5, mode=mode, gradient=gradient)
        else:
            c = _preference("", max(seqs // 2, 1), max(tokens, 2), mode=mode,
                            kind=rng.choice([SIGMOID, HINGE, SQUARED]),
                            beta=rng.choice([0.05, 0.1, 0.5, 2.0]), margin=rng.choice([0.0, 0.3]),
                            smoothing=rng.choice([0.0, 0.1]), reference=rng.random() < 0.7,
                            gradient=gradient)
    elif op in ("embed", "embed_grad"):
        hidden = _log_int(rng, 16, 8192)
        if rng.random() < 0.6:
            hidden = (hidden + 15) // 16 * 16
        # the largest listed table and batch bound the sizes
        vocab = _log_int(rng, 100, min(131072, 128256 * 4096 // (2 * hidden)))
        rows = _log_int(rng, 1, min(32768, 16384 * 4096 // (2 * hidden)))
        scale = rng.choice([1.0, math.sqrt(hidden)])
        c = (_embed if op == "embed" else _embed_grad)("", rows, hidden, vocab, dtype, out, scale)
    elif op == "act8":
        cols = _log_int(rng, 1, 14336)
        if rng.random() < 0.6:
            cols = (cols + 31) // 32 * 32
        c = _pack("", _log_int(rng, 1, min(16384, 8192 * 14336 // (2 * cols))), cols, dtype)
    else:
        cols, n = _log_int(rng, 64, 8192), _log_int(rng, 64, 14336)
        if rng.random() < 0.6:
            cols, n = (cols + 63) // 64 * 64, (n + 63) // 64 * 64
        most = min(16384, 8192 * 14336 * 4096 // (cols * n))
        c = _weight_grad("", _log_int(rng, 1, most), n, cols, out)
    del c["name"]
    return c


# -- inputs -------------------------------------------------------------------

def _torch_type(name):
    return torch.bfloat16 if name == "bf16" else torch.float32


def _seqs(case):
    return case["seqs"] if case["op"] == "policy" else 2 * case["pairs"]


def prepare(case, seed):
    dev = torch.device("cuda")
    gen = torch.Generator(device=dev).manual_seed(seed)
    st = {"case": case}
    {"policy": _prepare_sequences, "preference": _prepare_sequences, "embed": _prepare_embed,
     "embed_grad": _prepare_embed, "act8": _prepare_act8, "wgrad": _prepare_wgrad}[case["op"]](
         case, gen, dev, st)
    if own:
        _prepare_own(case, dev, st)
    return st


def _prepare_sequences(case, gen, dev, st):
    n, b = case["tokens"], _seqs(case)
    rand = lambda *s: torch.rand(*s, generator=gen, device=dev)
    randn = lambda *s: torch.randn(*s, generator=gen, device=dev)
    # packed sequences of different lengths, a few of them empty
    cuts = torch.sort((rand(b - 1) * n).long())[0]
    ends = torch.tensor([0, n], device=dev)
    st["offsets"] = torch.cat([ends[:1], cuts, ends[1:]])
    # a quarter of the positions are prompts, without a target
    tokens = torch.randint(0, 50304, (n,), generator=gen, device=dev)
    tokens[rand(n) < 0.25] = -1
    st["tokens"] = tokens
    # log probabilities of sampled tokens; the sampler's are an update older, the
    # reference's further away
    old = -torch.exp(randn(n) * 1.5 - 1.0)
    lp = torch.clamp(old + randn(n) * 0.2, max=0.0)
    st["logprob"] = lp
    st["ref"] = torch.clamp(lp + randn(n) * 0.3, max=0.0)
    if case["op"] == "policy":
        st["old"] = old
        st["advantage"] = randn(n if case["per_token"] else b)
        if case["kl_coef"] == 0.0:
            st["ref"] = None
        st["d_loss"] = torch.full((b,), 1.0 / (b if case["mode"] == MEAN else n), device=dev)
    else:
        if not case["reference"]:
            st["ref"] = None
        st["d_loss"] = torch.full((case["pairs"],), 1.0 / case["pairs"], device=dev)


def _prepare_embed(case, gen, dev, st):
    R, H, V = case["rows"], case["hidden"], case["vocab"]
    # token frequencies as in text: the k-th most frequent about 1 / k of the time
    u = torch.rand(R, generator=gen, device=dev, dtype=torch.float64)
    tokens = (torch.exp(u * math.log(V + 1.0)).long() - 1).clamp(0, V - 1)
    if R >= 64:
        tokens[torch.rand(R, generator=gen, device=dev) < 0.02] = -1      # padding
    st["tokens"] = tokens
    n = V if case["op"] == "embed" else R
    x = torch.empty(n, H, dtype=_torch_type(case["dtype"]), device=dev)
    for a in range(0, n, 16384):
        b = min(n, a + 16384)
        x[a:b] = torch.randn(b - a, H, generator=gen, device=dev) * 0.02
    st["x"] = x


def _activations(gen, dev, rows, cols):
    """Hidden activations: channels of different sizes, few of them large."""
    size = torch.exp(torch.randn(cols, generator=gen, device=dev) * 0.7)
    return torch.randn(rows, cols, generator=gen, device=dev) * size


def _prepare_act8(case, gen, dev, st):
    st["x"] = _activations(gen, dev, case["rows"], case["cols"]).to(_torch_type(case["dtype"]))


def _prepare_wgrad(case, gen, dev, st):
    T, C, N = case["rows"], case["cols"], case["out"]
    # what the forward pass has kept
    q, e = _plain_pack(_activations(gen, dev, T, C))
    st["q"], st["scale"] = q.contiguous(), e.contiguous()
    st["d_y"] = (torch.randn(T, N, generator=gen, device=dev) * 1e-3).to(torch.bfloat16)


def _prepare_own(case, dev, st):
    import fsdp_sharded_optimizer_flat_amd as z
    f = lambda *s: torch.empty(*s, device=dev)
    u8 = lambda *s: torch.empty(*s, dtype=torch.uint8, device=dev)
    op, o = case["op"], {}
    if op in ("policy", "preference"):
        b = _seqs(case)
        st["workspace"] = u8(z.zero_sequence_loss_workspace_bytes(case["tokens"], b))
        if op == "policy":
            o["loss"], o["kl"] = f(b), f(b) if st["ref"] is not None else None
            o["clipped"] = torch.empty(b, dtype=torch.int32, device=dev)
        else:
            o["loss"], o["reward"] = f(case["pairs"]), f(b)
        if case["gradient"]:
            o["d_logprob"] = f(case["tokens"])
    elif op == "embed":
        o["out"] = torch.empty(case["rows"], case["hidden"], dtype=_torch_type(case["out_dtype"]),
                               device=dev)
    elif op == "embed_grad":
        o["d_table"] = torch.empty(case["vocab"], case["hidden"],
                                   dtype=_torch_type(case["out_dtype"]), device=dev)
        st["workspace"] = u8(z.zero_embedding_grad_workspace_bytes(case["rows"], case["vocab"],
                                                                   case["hidden"]))
    elif op == "act8":
        R, C = case["rows"], case["cols"]
        st["q"], st["scale"] = u8(R, C), u8(R, (C + BLOCK - 1) // BLOCK)
        o["x"] = torch.empty_like(st["x"])
    else:
        o["d_w"] = torch.empty(case["out"], case["cols"], dtype=_torch_type(case["out_dtype"]),
                               device=dev)
        st["workspace"] = u8(z.zero_act8_weight_grad_workspace_bytes(case["rows"], case["out"],
                                                                     case["cols"]))
    st["output"] = o


# -- one pass --------------------------------------------------------------------

def run(st):
    return _run_own(st) if own else _PLAIN[st["case"]["op"]](st)


def _run_own(st):
    import fsdp_sharded_optimizer_flat_amd as z
    case, o = st["case"], st["output"]
    op = case["op"]
    if op in ("policy", "preference"):
        mode = z.ZERO_SEQUENCE_MEAN if case["mode"] == MEAN else z.ZERO_SEQUENCE_SUM
        d_loss = st["d_loss"] if case["gradient"] else None
    if op == "policy":
        z.zero_policy_loss(st["logprob"], st["old"], st["advantage"], st["offsets"],
                           tokens=st["tokens"], ref_logprob=st["ref"], per_token=case["per_token"],
                           clip_low=case["clip_low"], clip_high=case["clip_high"],
                           kl_coef=case["kl_coef"], mode=mode, d_loss=d_loss, loss=o["loss"],
                           kl=o["kl"], clipped=o["clipped"], d_logprob=o.get("d_logprob"),
                           workspace=st["workspace"])
    elif op == "preference":
        kind = {SIGMOID: z.ZERO_PREFER_SIGMOID, HINGE: z.ZERO_PREFER_HINGE,
                SQUARED: z.ZERO_PREFER_SQUARED}[case["kind"]]
        z.zero_preference_loss(st["logprob"], st["offsets"], tokens=st["tokens"],
                               ref_logprob=st["ref"], kind=kind, beta=case["beta"],
                               margin=case["margin"], mode=mode,
                               smoothing=case["smoothing"] if case["kind"] == SIGMOID else 0.0,
                               d_loss=d_loss, loss=o["loss"], reward=o["reward"],
                               d_logprob=o.get("d_logprob"), workspace=st["workspace"])
    elif op == "embed":
        z.zero_embedding(st["x"], st["tokens"], o["out"], scale=case["scale"])
    elif op == "embed_grad":
        z.zero_embedding_grad(st["x"], st["tokens"], o["d_table"], scale=case["scale"],
                              workspace=st["workspace"])
    elif op == "act8":
        z.zero_act8_pack(st["x"], st["q"], st["scale"])
        z.zero_act8_unpack(st["q"], st["scale"], o["x"])
    else:
        z.zero_act8_weight_grad(st["d_y"], st["q"], st["scale"], o["d_w"],
                                workspace=st["workspace"])
    return o


def _of_sequences(st):
    """Each token's sequence, and what sums values over each sequence."""
    off = st["offsets"]
    of = torch.repeat_interleave(torch.arange(off.numel() - 1, device=off.device),
                                 off[1:] - off[:-1], output_size=st["case"]["tokens"])

    def total(v):
        c = torch.cat([v.new_zeros(1), torch.cumsum(v, 0)])
        return c[off[1:]] - c[off[:-1]]
    return of, total


def _plain_policy(st):
    case = st["case"]
    on = st["tokens"] >= 0
    of, total = _of_sequences(st)
    lp = st["logprob"].double()
    adv = (st["advantage"] if case["per_token"] else st["advantage"][of]).double()
    ratio = torch.exp(lp - st["old"].double())
    free = -ratio * adv
    held = -ratio.clamp(1.0 - case["clip_low"], 1.0 + case["clip_high"]) * adv
    cut = on & (held > free)
    loss = torch.maximum(free, held)
    d = torch.where(cut, 0.0, free)
    o = {}
    kl = None
    if st["ref"] is not None:
        x = st["ref"].double() - lp
        kl = torch.expm1(x) - x
        loss = loss + case["kl_coef"] * kl
        d = d - case["kl_coef"] * torch.expm1(x)
    weight = torch.ones_like(total(lp))
    if case["mode"] == MEAN:
        weight = 1.0 / total(on.double()).clamp(min=1.0)
    o["loss"] = (total(torch.where(on, loss, 0.0)) * weight).float()
    o["kl"] = None if kl is None else (total(torch.where(on, kl, 0.0)) * weight).float()
    o["clipped"] = total(cut.double()).to(torch.int32)
    if case["gradient"]:
        o["d_logprob"] = torch.where(on, d * (weight * st["d_loss"].double())[of], 0.0).float()
    return o


def _plain_preference(st):
    case, pairs = st["case"], st["case"]["pairs"]
    on = st["tokens"] >= 0
    of, total = _of_sequences(st)
    term = st["logprob"].double()
    if st["ref"] is not None:
        term = term - st["ref"].double()
    score = total(torch.where(on, term, 0.0))
    weight = torch.ones_like(score)
    if case["mode"] == MEAN:
        weight = 1.0 / total(on.double()).clamp(min=1.0)
    reward = case["beta"] * score * weight
    h = reward[:pairs] - reward[pairs:] - case["margin"]
    if case["kind"] == SIGMOID:
        eps = case["smoothing"]
        grow = lambda v: v.clamp(min=0.0) + torch.log1p(torch.exp(-v.abs()))
        loss = (1.0 - eps) * grow(-h) + eps * grow(h)
        slope = eps / (1.0 + torch.exp(-h)) - (1.0 - eps) / (1.0 + torch.exp(h))
    elif case["kind"] == HINGE:
        loss = (1.0 - h).clamp(min=0.0)
        slope = torch.where(h < 1.0, -1.0, 0.0).double()
    else:
        loss = ((h - 0.5) / case["beta"]) ** 2
        slope = 2.0 * (h - 0.5) / case["beta"] ** 2
    o = {"loss": loss.float(), "reward": reward.float()}
    if case["gradient"]:
        d = st["d_loss"].double() * slope * case["beta"]
        d = torch.cat([d, -d]) * weight
        o["d_logprob"] = torch.where(on, d[of], 0.0).float()
    return o


def _plain_embed(st):
    case, t = st["case"], st["tokens"]
    rows = st["x"][t.clamp(min=0)].float() * case["scale"]
    return {"out": torch.where((t >= 0)[:, None], rows, 0.0).to(_torch_type(case["out_dtype"]))}


def _plain_embed_grad(st):
    case, t = st["case"], st["tokens"]
    d = torch.where((t >= 0)[:, None], st["x"].float(), 0.0)
    g = torch.zeros(case["vocab"], case["hidden"], device=t.device)
    g.index_add_(0, t.clamp(min=0), d)
    return {"d_table": (g * case["scale"]).to(_torch_type(case["out_dtype"]))}


def _blocks(x):
    """(rows, blocks, 32), the last block filled up with zeros."""
    rows, cols = x.shape
    n = (cols + BLOCK - 1) // BLOCK
    full = x.new_zeros(rows, n * BLOCK)
    full[:, :cols] = x
    return full.view(rows, n, BLOCK)


def _plain_pack(x):
    """The codes (e4m3) of x and their blocks' scales: the least power of two
    that brings the block's largest magnitude to 448 or less, as its exponent
    + 127."""
    cols = x.shape[1]
    x = _blocks(x.float())
    m, e = torch.frexp(x.abs().amax(2))                  # m in [1/2, 1): 448 = 0.875 * 2^9
    e = torch.where(m > 0.875, e - 8, e - 9).clamp(min=-127)
    e = torch.where(m == 0, -127, e)
    q = torch.ldexp(x, -e[..., None]).to(torch.float8_e4m3fn).view(torch.uint8)
    return q.flatten(1)[:, :cols], (e + 127).to(torch.uint8)


def _plain_unpack(q, scale):
    cols = q.shape[1]
    x = _blocks(q).view(torch.float8_e4m3fn).float()
    return torch.ldexp(x, (scale.int() - 127)[..., None]).flatten(1)[:, :cols]


def _plain_act8(st):
    return {"x": _plain_unpack(*_plain_pack(st["x"])).to(st["x"].dtype)}


def _plain_wgrad(st):
    d = st["d_y"].float().t() @ _plain_unpack(st["q"], st["scale"])
    return {"d_w": d.to(_torch_type(st["case"]["out_dtype"]))}


_PLAIN = {"policy": _plain_policy, "preference": _plain_preference, "embed": _plain_embed,
          "embed_grad": _plain_embed_grad, "act8": _plain_act8, "wgrad": _plain_wgrad}


# -- what a pass cannot do without ---------------------------------------------------

def _size(name):
    return 2 if name == "bf16" else 4


def work(case):
    op = case["op"]
    if op in ("policy", "preference"):
        n, b = float(case["tokens"]), _seqs(case)
        if op == "policy":
            kl = case["kl_coef"] != 0.0
            byt = n * (8 + 4 + 4 + 4 * kl + 4 * case["gradient"])
            byt += 4.0 * (n if case["per_token"] else b) + 8.0 * b + 4.0 * b * (2 + kl)
            return {"bytes": byt + 4.0 * b * case["gradient"], "flops": n * (10.0 + 10.0 * kl)}
        byt = n * (8 + 4 + 4 * case["reference"] + 4 * case["gradient"])
        return {"bytes": byt + 16.0 * b, "flops": 2.0 * n}
    if op == "embed":
        n = float(case["rows"]) * case["hidden"]
        # rows of tokens that repeat are read once: about these many differ
        k, v = case["rows"], case["vocab"]
        differ = sum(1.0 - (1.0 - 1.0 / ((i + 1.0) * math.log(v + 1.0))) ** k for i in range(v))
        return {"bytes": differ * case["hidden"] * _size(case["dtype"]) +
                n * _size(case["out_dtype"]) + 8.0 * k, "flops": n}
    if op == "embed_grad":
        n = float(case["rows"]) * case["hidden"]
        return {"bytes": n * _size(case["dtype"]) + 8.0 * case["rows"] +
                float(case["vocab"]) * case["hidden"] * _size(case["out_dtype"]), "flops": 2.0 * n}
    if op == "act8":
        # values in, codes and scales out and in again, values out
        n = float(case["rows"]) * case["cols"]
        return {"bytes": 2.0 * n * (_size(case["dtype"]) + 1.0 + 1.0 / BLOCK), "flops": 6.0 * n}
    T, C, N = float(case["rows"]), case["cols"], case["out"]
    return {"bytes": T * (2.0 * N + C * (1.0 + 1.0 / BLOCK)) + float(N) * C * _size(case["out_dtype"]),
            "flops": 2.0 * T * N * C}


# -- the definition in 64 bits -----------------------------------------------------------

def exact(case, seed):
    global own
    kept, own = own, False
    try:
        st = prepare(case, seed)
    finally:
        own = kept
    return _EXACT[case["op"]](case, st)


def _each_sequence(st):
    """Each token's sequence by search, and what sums values over each sequence."""
    off, n = st["offsets"], st["case"]["tokens"]
    where = torch.searchsorted(off, torch.arange(n, device=off.device), right=True) - 1

    def sums(v):
        # a thousand running totals a sequence, so that few additions meet
        b, lanes = off.numel() - 1, max(1, min(1024, (1 << 22) // off.numel()))
        at = where * lanes + torch.arange(n, device=off.device) % lanes
        return v.new_zeros(b * lanes).scatter_add(0, at, v).view(b, lanes).sum(1)
    return where, sums


def _exact_policy(case, st):
    f64 = torch.float64
    where, sums = _each_sequence(st)
    target = (st["tokens"] >= 0).to(f64)
    a = st["advantage"].to(f64)
    a = a if case["per_token"] else a.take(where)
    step = st["logprob"].to(f64) - st["old"].to(f64)
    # a positive advantage is cut above the upper border, a negative one below the lower
    beyond = torch.where(a > 0, step > math.log1p(case["clip_high"]),
                         (a < 0) & (step < math.log1p(-case["clip_low"])))
    border = torch.where(a > 0, 1.0 + case["clip_high"], 1.0 - case["clip_low"]).to(f64)
    value = -a * torch.where(beyond, border, step.exp())
    slope = -a * torch.where(beyond, torch.zeros_like(step), step.exp())
    count = sums(target)
    share = torch.ones_like(count) if case["mode"] == SUM else count.clamp(min=1).reciprocal()
    out = {"kl": None}
    if st["ref"] is not None:
        gap = st["ref"].to(f64) - st["logprob"].to(f64)
        k = torch.special.expm1(gap) - gap
        value = value + k * case["kl_coef"]
        slope = slope - torch.special.expm1(gap) * case["kl_coef"]
        out["kl"] = sums(k * target) * share
    out["loss"] = sums(value * target) * share
    out["clipped"] = sums(beyond * target).round().to(torch.int32)
    if case["gradient"]:
        out["d_logprob"] = slope * target * (share * st["d_loss"].to(f64)).take(where)
    return {k: out[k] for k in ("loss", "kl", "clipped", "d_logprob") if k in out}


def _exact_preference(case, st):
    f64, P = torch.float64, case["pairs"]
    where, sums = _each_sequence(st)
    target = (st["tokens"] >= 0).to(f64)
    t = st["logprob"].to(f64) - (0.0 if st["ref"] is None else st["ref"].to(f64))
    share = 1.0 if case["mode"] == SUM else 1.0 / sums(target).clamp(min=1)
    reward = sums(t * target) * share * case["beta"]
    h = (reward[:P] - reward[P:] - case["margin"]).requires_grad_()
    with torch.enable_grad():
        if case["kind"] == SIGMOID:
            s = case["smoothing"]
            loss = -(1 - s) * torch.nn.functional.logsigmoid(h) - s * torch.nn.functional.logsigmoid(-h)
        elif case["kind"] == HINGE:
            loss = torch.relu(1 - h)
        else:
            loss = ((h / case["beta"]) - 1 / (2 * case["beta"])).square()
        dh, = torch.autograd.grad(loss.sum(), h)
    out = {"loss": loss.detach(), "reward": reward}
    if case["gradient"]:
        g = dh * st["d_loss"].to(f64) * case["beta"]
        g = torch.cat((g, -g)) * share
        out["d_logprob"] = g.take(where) * target
    return out


def _exact_embed(case, st):
    t = st["tokens"]
    out = torch.zeros(case["rows"], case["hidden"], dtype=torch.float64, device=t.device)
    keep = t.ge(0).nonzero()[:, 0]
    out[keep] = st["x"].index_select(0, t[keep]).to(torch.float64) * case["scale"]
    return {"out": out}


def _exact_embed_grad(case, st):
    t, x = st["tokens"], st["x"]
    order = torch.argsort(t, stable=True)
    order = order[t[order] >= 0]
    ids, counts = torch.unique_consecutive(t[order], return_counts=True)
    out = torch.zeros(case["vocab"], case["hidden"], dtype=torch.float64, device=t.device)
    ends = torch.cumsum(counts, 0)
    # differences of running sums, some columns at a time
    for a in range(0, case["hidden"], 256):
        c = torch.cumsum(x[order, a:a + 256].to(torch.float64), 0)
        c = torch.cat([torch.zeros_like(c[:1]), c])
        out[ids, a:a + 256] = (c[ends] - c[ends - counts]) * case["scale"]
    return {"d_table": out}


def _nearest_code(v):
    """v rounded to four significant bits, ties to even, with e4m3's least step 2^-9."""
    step = torch.exp2(torch.floor(torch.log2(v.abs().clamp(min=2.0 ** -6))) - 3.0)
    return torch.round(v / step) * step


def _exact_act8(case, st):
    x = st["x"].to(torch.float64)
    out = torch.empty_like(x)
    for a in range(0, case["cols"], BLOCK):
        part = x[:, a:a + BLOCK]
        top = part.abs().amax(1, keepdim=True)
        e = torch.ceil(torch.log2((top / 448.0).clamp(min=2.0 ** -127)))
        e = torch.where(top > 448.0 * torch.exp2(e), e + 1, e)
        e = torch.where((e > -127) & (top <= 448.0 * torch.exp2(e - 1)), e - 1, e)
        out[:, a:a + BLOCK] = _nearest_code(part * torch.exp2(-e)) * torch.exp2(e)
    return {"x": out}


def _exact_wgrad(case, st):
    codes = torch.arange(256, device="cuda")
    power, low = (codes >> 3) & 15, (codes & 7).to(torch.float64)
    value = torch.where(power > 0, (8.0 + low) * torch.exp2(power - 10.0), low * 2.0 ** -9)
    value = torch.where(codes >= 128, -value, value)
    x = value[st["q"].int()]
    scale = torch.exp2(st["scale"].to(torch.float64) - 127.0)
    x = x * scale.repeat_interleave(BLOCK, 1)[:, :case["cols"]]
    return {"d_w": torch.matmul(st["d_y"].to(torch.float64).T, x)}


_EXACT = {"policy": _exact_policy, "preference": _exact_preference, "embed": _exact_embed,
          "embed_grad": _exact_embed_grad, "act8": _exact_act8, "wgrad": _exact_wgrad}
