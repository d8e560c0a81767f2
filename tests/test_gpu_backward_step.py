"""The operators around the token losses as a training step uses them, on the GPU:
embedding, checkpoints, log probabilities, a loss over sequences, the gradients of
head, projection and embedding in one unit's bucket, the sharded optimizer step, the
next step's weights; a bad token that skips the clipped step; the calls captured in
a graph, and side by side on host threads with streams of their own.

Each operator's result is checked against binary64 on its own inputs (tolerances of
its own test file); the optimizer step against the oracle, bit for bit, from the very
buckets that the gradients went into."""
import threading

import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():
    pytest.skip("needs a GPU", allow_module_level=True)

import act8_ref  # noqa: E402
import oracle  # noqa: E402
import sequence_ref  # noqa: E402
import fsdp_sharded_optimizer_flat_amd as z  # noqa: E402
from gpu_common import DEV, assert_same_bf16, assert_same_f32, hyper_args, scalars, to_np  # noqa: E402

G, Lc = z.ZERO_GLOBAL, z.ZERO_LOCAL
H = dict(lr=1e-2, b1=0.9, b2=0.95, eps=1e-8, wd=0.1)
N, TOKENS, VOCAB, WIDTH = 3, 200, 2003, 96
OFFSETS = [0, 70, 70, 151, 200]
BF16, F32 = 2.0 ** -8, 2.0 ** -24


def bytes_of(n):
    return torch.full((max(n, 16),), 255, dtype=torch.uint8, device=DEV)


class Model:
    """logits = (E[tokens] scale W^T) E^T: a tied embedding E and a projection W as the
    one unit of a layout over N ranks, every rank's shard on this device."""

    scale = 2.0

    def __init__(self, seed):
        g = torch.Generator(device=DEV).manual_seed(seed)
        self.numel = [VOCAB * WIDTH + WIDTH * WIDTH]
        self.L = z.zero_pack(N, self.numel)
        self.master = torch.zeros(self.L.padded, device=DEV)
        self.master[:self.numel[0]] = torch.randn(self.numel[0], generator=g, device=DEV) * 0.2
        self.m, self.v = torch.zeros_like(self.master), torch.zeros_like(self.master)
        self.out = self.master.to(torch.bfloat16).view(torch.int16).clone()
        self.buckets = [torch.zeros(self.L.padded, dtype=torch.bfloat16, device=DEV) for _ in range(N)]
        ri = lambda: torch.randint(0, VOCAB, (TOKENS,), generator=g, device=DEV)
        self.tokens, self.targets = [ri() for _ in range(N)], [ri() for _ in range(N)]
        for r in range(N):
            self.tokens[r][::3] = 7           # one token of many rows
            self.targets[r][:20] = -1         # a prompt
        self.noise = [torch.randn(2, TOKENS, generator=g, device=DEV) * 0.2 for _ in range(N)]
        self.advantage = [torch.randn(4, generator=g, device=DEV) for _ in range(N)]
        self.offsets = torch.tensor(OFFSETS, device=DEV)
        self.d_loss = torch.full((4,), 0.25, device=DEV)

    def parts(self, flat):
        k = VOCAB * WIDTH
        return flat[:k].view(VOCAB, WIDTH), flat[k:self.numel[0]].view(WIDTH, WIDTH)

    def weights(self):
        return self.parts(self.out.view(torch.bfloat16))

    def forward(self, r):
        """What the backward pass needs: checkpoints, logits, log probabilities."""
        E, W = self.weights()
        f = {"x": torch.empty(TOKENS, WIDTH, dtype=torch.bfloat16, device=DEV)}
        z.zero_embedding(E, self.tokens[r], f["x"], scale=self.scale)
        f["y"] = torch.mm(f["x"], W.t())
        for k in "xy":
            f[k + "8"] = (torch.empty(TOKENS, WIDTH, dtype=torch.uint8, device=DEV),
                          torch.empty(TOKENS, WIDTH // 32, dtype=torch.uint8, device=DEV))
            z.zero_act8_pack(f[k], *f[k + "8"])
        f["logits"] = torch.mm(f["y"], E.t())
        f["lp"], f["stats"] = torch.empty(TOKENS, device=DEV), torch.empty(TOKENS, 2, device=DEV)
        z.zero_logprob(f["logits"], self.targets[r], logprob=f["lp"], stats=f["stats"],
                       workspace=bytes_of(z.zero_loss_workspace_bytes(TOKENS, VOCAB)))
        f["old"], f["ref"] = f["lp"] + self.noise[r][0], f["lp"] + self.noise[r][1]
        return f

    def loss(self, r, f):
        f["loss"], f["d_lp"] = torch.empty(4, device=DEV), torch.full((TOKENS,), 9.0, device=DEV)
        z.zero_policy_loss(f["lp"], f["old"], self.advantage[r], self.offsets, tokens=self.targets[r],
                           ref_logprob=f["ref"], kl_coef=0.1, d_loss=self.d_loss, loss=f["loss"], d_logprob=f["d_lp"],
                           workspace=bytes_of(z.zero_sequence_loss_workspace_bytes(TOKENS, 4)))
        f["d_logits"] = torch.empty_like(f["logits"])
        z.zero_logprob_grad(f["logits"], self.targets[r], f["stats"], f["d_logits"], d_logprob=f["d_lp"])

    def backward(self, r, f):
        E, W = self.weights()
        d_E, d_W = self.parts(self.buckets[r])
        ws = lambda o: bytes_of(z.zero_act8_weight_grad_workspace_bytes(TOKENS, o, WIDTH))
        z.zero_act8_weight_grad(f["d_logits"], *f["y8"], d_E, workspace=ws(VOCAB))
        f["head"] = d_E.clone()
        f["d_y"] = torch.mm(f["d_logits"], E)
        z.zero_act8_weight_grad(f["d_y"], *f["x8"], d_W, workspace=ws(WIDTH))
        f["d_x"] = torch.mm(f["d_y"], W)
        z.zero_embedding_grad(f["d_x"], self.tokens[r], d_E, scale=self.scale, accumulate=True,
                              workspace=bytes_of(z.zero_embedding_grad_workspace_bytes(TOKENS, VOCAB, WIDTH)))

    def check(self, r, f, E):
        """Each operator against binary64 on the inputs it had."""
        D = lambda t: t.double()
        within = lambda got, want, tol: bool(((D(got) - want).abs() <= tol).all())
        want = D(E)[self.tokens[r]] * self.scale
        assert within(f["x"], want, want.abs() * BF16)
        kept = {}
        for k in "xy":
            byte, kept[k] = act8_ref.pack_values(f[k])
            assert torch.equal(f[k + "8"][1].cpu().long(), byte)
            assert torch.equal(act8_ref.unpack_values(*f[k + "8"]), kept[k])
            kept[k] = kept[k].to(DEV)
        n = lambda t: t.cpu().numpy()
        loss, _, _, d_lp = sequence_ref.policy(n(f["lp"]), n(f["old"]), n(f["ref"]), n(self.advantage[r]), False,
                                               n(self.targets[r]), OFFSETS, 0.2, 0.2, 0.1, "mean", n(self.d_loss),
                                               np.full(TOKENS, 9.0))
        assert np.all(np.abs(n(f["loss"]) - loss) <= np.abs(loss) * F32 + 1e-11)
        assert np.all(np.abs(n(f["d_lp"]) - d_lp) <= 2 * np.abs(d_lp) * F32 + 1e-11)
        for got, d_y, x, was in ((f["head"], f["d_logits"], kept["y"], None),
                                 (self.parts(self.buckets[r])[1], f["d_y"], kept["x"], None)):
            want, size = D(d_y).T @ x, D(d_y).abs().T @ x.abs()
            err = TOKENS * 2.0 ** -23 * size
            assert within(got, want, err + (want.abs() + err) * BF16)
        add = torch.zeros(VOCAB, WIDTH, dtype=torch.float64, device=DEV)
        size = torch.zeros_like(add)
        for t in range(TOKENS):
            add[self.tokens[r][t]] += D(f["d_x"][t]) * self.scale
            size[self.tokens[r][t]] += D(f["d_x"][t]).abs() * self.scale
        want = D(f["head"]) + add
        err = TOKENS * F32 * size + (want.abs() + size) * 2 * F32
        got = self.parts(self.buckets[r])[0]
        assert within(got, want, err + (want.abs() + err) * BF16)
        untouched = torch.ones(VOCAB, dtype=torch.bool, device=DEV)
        untouched[self.tokens[r]] = False
        assert torch.equal(got[untouched], f["head"][untouched])


def test_policy_steps():
    model = Model(1)
    want = [to_np(t).copy() for t in (model.master, model.m, model.v, model.out)]
    for t in (1, 2):
        for r in range(N):
            f = model.forward(r)
            model.loss(r, f)
            model.backward(r, f)
            torch.cuda.synchronize()
            model.check(r, f, model.weights()[0])
        z.zero_step_units(model.L, -1, 0, 1, model.buckets, G, float(N), model.master, model.m, model.v, G, model.out,
                          G, scalars(t, H))
        torch.cuda.synchronize()
        oracle.zero_step_all(N, model.numel, [np.ascontiguousarray(to_np(b)) for b in model.buckets], divisor=float(N),
                             clip=1.0, master=want[0], m=want[1], v=want[2], out=want[3], t=t, **hyper_args(H))
        for got, w, name in zip((model.master, model.m, model.v), want, ("master", "m", "v")):
            assert_same_f32(to_np(got), w, f"step {t} {name}")
        assert_same_bf16(to_np(model.out), want[3], f"step {t} out")


@pytest.mark.parametrize("where", ["target", "embedding"])
def test_a_bad_token_skips_the_clipped_step(where):
    """A token past the vocabulary, as a target or as an input, reaches the buckets as
    NaN: the clip coefficient is NaN and the step leaves the state as it was."""
    model = Model(2)
    for r in range(N):
        (model.targets if where == "target" else model.tokens)[r][150] = VOCAB
        f = model.forward(r)
        model.loss(r, f)
        assert bool(f["loss"].isnan().any()) and bool(f["d_logits"][150].isnan().all())
        model.backward(r, f)
    before = [t.clone() for t in (model.master, model.m, model.v, model.out)]
    ws = torch.zeros(z.zero_gradnorm_workspace_bytes(model.L, -1) // 8, dtype=torch.float64, device=DEV)
    sumsq, coef = torch.zeros(1, dtype=torch.float64, device=DEV), torch.zeros(1, device=DEV)
    z.zero_gradnorm_async(model.L, -1, model.buckets, G, float(N), None, G, ws, sumsq)
    z.zero_clip_coef_async(sumsq, 1.0, coef)
    z.zero_step_device_clip(model.L, -1, model.buckets, G, float(N), model.master, model.m, model.v, G, model.out, G,
                            scalars(1, H), coef)
    torch.cuda.synchronize()
    assert bool(coef.isnan().all())
    for a, b in zip(before, (model.master, model.m, model.v, model.out)):
        assert torch.equal(a, b)


def test_losses_through_the_logits_against_autograd():
    """d(loss) / d(logits) of both losses, through zero_logprob_grad, against torch's own
    derivative of the whole formula in binary64 on the host."""
    model = Model(3)
    f = model.forward(0)
    targets = model.targets[0].cpu()
    on = targets >= 0
    spans = list(zip(OFFSETS[:-1], OFFSETS[1:]))
    x = f["logits"].double().cpu().requires_grad_()
    lp = torch.log_softmax(x, 1).gather(1, targets.clamp(min=0)[:, None])[:, 0]
    old, ref, adv = (t.double().cpu() for t in (f["old"], f["ref"], model.advantage[0]))
    for kind in ("policy", "preference"):
        if kind == "policy":
            ratio = torch.exp(lp - old)
            a = torch.cat([adv[i].expand(hi - lo) for i, (lo, hi) in enumerate(spans)])
            term = torch.maximum(-ratio * a, -ratio.clamp(0.8, 1.2) * a)
            gap = ref - lp
            term = term + 0.1 * (torch.exp(gap) - 1 - gap)
            total = 0.25 * sum(term[lo:hi][on[lo:hi]].mean() for lo, hi in spans if on[lo:hi].any())
            model.loss(0, f)
        else:
            s = [0.3 * (lp - ref)[lo:hi][on[lo:hi]].sum() for lo, hi in spans]
            total = sum(torch.nn.functional.softplus(s[p + 2] - s[p]) * 0.5 for p in range(2))
            d_lp, half = torch.zeros(TOKENS, device=DEV), torch.full((2,), 0.5, device=DEV)
            z.zero_preference_loss(f["lp"], model.offsets, tokens=model.targets[0], ref_logprob=f["ref"], beta=0.3,
                                   d_loss=half, d_logprob=d_lp, loss=torch.empty(2, device=DEV),
                                   workspace=bytes_of(z.zero_sequence_loss_workspace_bytes(TOKENS, 4)))
            f["d_logits"] = torch.empty_like(f["logits"])
            z.zero_logprob_grad(f["logits"], model.targets[0], f["stats"], f["d_logits"], d_logprob=d_lp)
        want, = torch.autograd.grad(total, x, retain_graph=True)
        got = f["d_logits"].double().cpu()
        # the log probabilities the losses start from are binary32 (2^-22 of values up to
        # 16 or so), which moves ratios and k's slopes by 2^-18 of themselves at most;
        # probabilities likewise; then one rounding to bf16
        size = want.abs().amax(1, keepdim=True)
        assert bool(((got - want).abs() <= want.abs() * BF16 + size * 2.0 ** -14).all()), kind


def test_a_graph_of_the_backward_pass():
    """All of the pass but the library's products, captured once and replayed between
    eager passes over other inputs."""
    model = Model(4)
    f = model.forward(0)
    model.loss(0, f)
    model.backward(0, f)
    kept = {k: bytes_of(n) for k, n in (("loss", z.zero_loss_workspace_bytes(TOKENS, VOCAB)),
                                        ("seq", z.zero_sequence_loss_workspace_bytes(TOKENS, 4)),
                                        ("head", z.zero_act8_weight_grad_workspace_bytes(TOKENS, VOCAB, WIDTH)),
                                        ("proj", z.zero_act8_weight_grad_workspace_bytes(TOKENS, WIDTH, WIDTH)),
                                        ("emb", z.zero_embedding_grad_workspace_bytes(TOKENS, VOCAB, WIDTH)))}
    ins = {k: f[k].clone() for k in ("x", "y", "logits", "old", "ref", "d_y", "d_x")}
    E = model.weights()[0].clone()

    def run(i, ws):
        o = {k: torch.empty(TOKENS, device=DEV) for k in ("lp", "d_lp")}
        o["stats"], o["loss"] = torch.empty(TOKENS, 2, device=DEV), torch.empty(4, device=DEV)
        o["d_logits"], o["x"] = torch.empty_like(i["logits"]), torch.empty_like(i["x"])
        o["d_E"] = torch.empty(VOCAB, WIDTH, dtype=torch.bfloat16, device=DEV)
        o["d_W"] = torch.empty(WIDTH, WIDTH, dtype=torch.bfloat16, device=DEV)
        q = {k: (torch.empty(TOKENS, WIDTH, dtype=torch.uint8, device=DEV),
                 torch.empty(TOKENS, WIDTH // 32, dtype=torch.uint8, device=DEV)) for k in "xy"}

        def calls():
            z.zero_embedding(E, model.tokens[0], o["x"], scale=2.0)
            for k in "xy":
                z.zero_act8_pack(i[k], *q[k])
            z.zero_logprob(i["logits"], model.targets[0], logprob=o["lp"], stats=o["stats"], workspace=ws["loss"])
            z.zero_policy_loss(o["lp"], i["old"], model.advantage[0], model.offsets, tokens=model.targets[0],
                               ref_logprob=i["ref"], kl_coef=0.1, d_loss=model.d_loss, loss=o["loss"],
                               d_logprob=o["d_lp"], workspace=ws["seq"])
            z.zero_logprob_grad(i["logits"], model.targets[0], o["stats"], o["d_logits"], d_logprob=o["d_lp"])
            z.zero_act8_weight_grad(o["d_logits"], *q["y"], o["d_E"], workspace=ws["head"])
            z.zero_act8_weight_grad(i["d_y"], *q["x"], o["d_W"], workspace=ws["proj"])
            z.zero_embedding_grad(i["d_x"], model.tokens[0], o["d_E"], scale=2.0, accumulate=True,
                                  workspace=ws["emb"])
        return o, calls

    out, calls = run(ins, kept)
    calls()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        calls()
    g = torch.Generator(device=DEV).manual_seed(5)
    for turn in range(4):
        for k in ins:
            ins[k].copy_(f[k].float() * (1.0 + 0.2 * torch.rand(f[k].shape, generator=g, device=DEV)))
        want, eager = run({k: v.clone() for k, v in ins.items()}, {k: torch.empty_like(v) for k, v in kept.items()})
        eager()
        torch.cuda.synchronize()
        for v in out.values():
            v.fill_(3)
        graph.replay()
        torch.cuda.synchronize()
        for k in out:
            assert torch.equal(out[k], want[k]), (turn, k)


def test_four_threads_on_streams_of_their_own():
    models = [Model(10 + i) for i in range(4)]

    def run(model):
        for r in range(N):
            f = model.forward(r)
            model.loss(r, f)
            model.backward(r, f)

    for m in models:
        run(m)
    torch.cuda.synchronize()
    want = [[b.clone() for b in m.buckets] for m in models]
    for m in models:
        for b in m.buckets:
            b.zero_()
    torch.cuda.synchronize()
    failed = []

    def work(model, stream):
        try:
            with torch.cuda.stream(stream):
                run(model)
            stream.synchronize()
        except Exception as e:   # noqa: BLE001  (reported by the main thread)
            failed.append(e)

    threads = [threading.Thread(target=work, args=(m, torch.cuda.Stream())) for m in models]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not failed, failed
    for m, w in zip(models, want):
        for got, b in zip(m.buckets, w):
            assert torch.equal(got, b)
