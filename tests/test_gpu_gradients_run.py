"""The operators that make the gradients together, as a training step uses
them: a run checked against autograd in 64 bits and fed to the optimizer's
operators; captured and replayed; on other streams; from several host threads;
past 2^32 bytes."""
import threading

import pytest
import torch

import quantized_momentum_newton_amd as q
from gpu_util import say

pytestmark = pytest.mark.gpu
DEV = "cuda"
B, F = torch.bfloat16, torch.float32


class Block:
    """embedding -> gated feed-forward -> linear loss; bf16 compute weights,
    gradients in fp32 buffers."""

    def __init__(self, vocab=300, width=128, hidden=272, tokens=200, act="silu", seed=0):
        gen = torch.Generator(device=DEV).manual_seed(seed)
        new = lambda *s, std: torch.randn(*s, generator=gen, device=DEV) * std
        self.act, self.hidden, self.scale = act, hidden, width ** 0.5
        self.table = new(vocab, width, std=0.1)
        self.wgu = new(2 * hidden, width, std=width ** -0.5).to(B)
        self.wd = new(width, hidden, std=hidden ** -0.5).to(B)
        self.tokens = torch.randint(-1, vocab, (tokens,), generator=gen, device=DEV)
        self.r = new(tokens, width, std=1e-2).to(B)
        self.grads = [torch.empty_like(self.table), torch.empty(2 * hidden, width, device=DEV), torch.empty(width, hidden, device=DEV)]
        self.ws = [q.embedding_grad_workspace(self.tokens, self.r, self.grads[0]),
                   torch.empty(max(1, q.weight_grad_workspace_bytes(tokens, 2 * hidden, width),
                                   q.weight_grad_workspace_bytes(tokens, width, hidden)), dtype=torch.uint8, device=DEV)]

    def step(self, accumulate=False):
        """The loss is sum(r * y); its gradients, in the buffers."""
        de, dgu, dd = self.grads
        n = self.hidden
        x = q.embedding_lookup(self.tokens, self.table, self.scale, dtype=B)
        x8 = q.act_pack(x)
        gu = x @ self.wgu.t()
        h, g8, u8 = q.gated_act_forward(gu[:, :n], gu[:, n:], act=self.act)
        y = h @ self.wd.t()
        dh = self.r @ self.wd
        dgu_out = torch.empty_like(gu)
        _, _, again = q.gated_act_backward(g8, u8, dh, dgu_out[:, :n], dgu_out[:, n:], recompute=True, act=self.act)
        q.weight_grad(self.r, again, dd, accumulate=accumulate, ws=self.ws[1])
        q.weight_grad(dgu_out, x8, dgu, accumulate=accumulate, ws=self.ws[1])
        dx = dgu_out @ self.wgu
        q.embedding_grad(self.tokens, dx, de, self.scale, accumulate=accumulate, ws=self.ws[0])
        return y

    def reference(self):
        """autograd in 64 bits, nothing kept in 8."""
        t, wgu, wd = (w.detach().double().cpu().requires_grad_() for w in (self.table, self.wgu, self.wd))
        tok = self.tokens.cpu()
        x = t[tok.clamp(min=0)] * self.scale * (tok >= 0)[:, None]
        g, u = (x @ wgu.t()).split(self.hidden, 1)
        a = torch.nn.functional.silu(g) if self.act == "silu" else torch.nn.functional.gelu(g, approximate="tanh")
        y = (a * u) @ wd.t()
        (y * self.r.double().cpu()).sum().backward()
        return y, [t.grad, wgu.grad, wd.grad]


@pytest.mark.parametrize("act", ["silu", "gelu"])
@pytest.mark.parametrize("sizes", [dict(), dict(vocab=57, width=100, hidden=77, tokens=333), dict(width=256, hidden=640, tokens=2100)])
def test_a_training_step_against_autograd(act, sizes):
    """y comes from unquantised activations: bf16 roundings of four stages, each
    2^-9 of its values, through sums of random signs (3 * 2^-7 allowed).  The
    gradients take up to three factors from 8 bits, each off by at most 1/16 of
    itself and by a third of that in the mean square, so by less than 3/16."""
    m = Block(act=act, **sizes)
    y = m.step()
    want_y, want = m.reference()
    rel = lambda a, b: ((a.double().cpu() - b).norm() / b.norm()).item()
    assert rel(y, want_y) < 3 * 2.0 ** -7
    for got, exact, name in zip(m.grads, want, ("embedding", "gate and up", "down")):
        say(name, rel(got, exact))
        assert rel(got, exact) < 3 / 16, name
    once = [g.clone() for g in m.grads]
    m.step(accumulate=True)
    for g, o in zip(m.grads, once):
        assert torch.equal(g, 2 * o)


def test_gradients_go_to_the_optimizer():
    """The buffers as a gradient list, Muon's matrices and AdamW's table."""
    m = Block()
    plan = q.GradPlan(m.grads)
    weights = [m.table, m.wgu.float(), m.wd.float()]
    codes = [torch.zeros(w.numel(), dtype=torch.int8, device=DEV) for w in weights[1:]]
    absmax = [torch.zeros(-(-w.numel() // 256), device=DEV) for w in weights[1:]]
    mats = [(*w.shape, *w.shape, w) for w in weights[1:]]
    muon = q.Plan([(c, a, g.view(-1)) for c, a, g in zip(codes, absmax, m.grads[1:])],
                  [(i, 0, w.numel(), i) for i, w in enumerate(weights[1:])], 2)
    adamw = q.AdamWPlan([(m.table, m.grads[0], q.AdamWState(m.table.numel(), bits=8, device=DEV), None, 1.0, 0.0)])
    before = [w.clone() for w in weights]
    m.step()
    norm, coef = q.grad_norm(plan, 0.01)
    exact = sum(g.double().square().sum().item() for g in m.grads) ** 0.5
    assert abs(norm.item() / exact - 1) < 2.0 ** -22
    q.grad_scale(plan, coef)
    q.muon_step(muon, None, mats, 1, q.make_hparams(period=1))
    q.adamw_step(adamw, 1, lr=1e-3)
    torch.cuda.synchronize()
    for w, b in zip(weights, before):
        assert torch.isfinite(w).all() and not torch.equal(w, b)
    rows = torch.zeros(len(m.table), dtype=torch.bool, device=DEV)
    rows[m.tokens[m.tokens >= 0]] = True
    assert torch.equal(m.table[~rows], before[0][~rows])      # no token, no gradient, no decay


def test_captured_and_replayed():
    """One graph of the whole step, replayed on new inputs with eager work in
    between, and a second graph that shares its workspaces, bit for bit."""
    m, other = Block(tokens=1500, width=64, hidden=96), Block(tokens=1500, width=64, hidden=96, seed=5)
    other.ws = m.ws
    side = torch.cuda.Stream()
    graphs = []
    for b in (m, other):
        b.step()                     # kernels are loaded before a capture
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=side):
            y = b.step(accumulate=True)
        graphs.append((b, g, y))
    for seed in range(3):
        gen = torch.Generator(device=DEV).manual_seed(100 + seed)
        for b, g, y in graphs:
            b.tokens.copy_(torch.randint(-1, 300, b.tokens.shape, generator=gen, device=DEV))
            b.r.copy_(torch.randn(b.r.shape, generator=gen, device=DEV) * 1e-2)
            for w in b.ws:
                w.fill_(seed * 85)
            for d in b.grads:
                d.fill_(0.5)
            g.replay()
            got = [y.clone()] + [d.clone() for d in b.grads]
            for d in b.grads:
                d.fill_(0.5)
            want = [b.step(accumulate=True)] + b.grads
            torch.cuda.synchronize()
            for a, c in zip(got, want):
                assert torch.equal(a, c)
    say("replays equal")


def test_given_stream():
    """Inputs written and results read on the given stream, outputs and
    workspaces made by the calls."""
    side = torch.cuda.Stream()
    x = torch.randn(300, 96, device=DEV).to(B)
    up = torch.randn(300, 96, device=DEV).to(B)
    tok = torch.randint(0, 50, (300,), device=DEV)
    table = torch.randn(50, 96, device=DEV)

    def run(stream):
        c = q.act_pack(x, stream=stream)
        h, g8, u8 = q.gated_act_forward(x, up, stream=stream)
        dg, du, again = q.gated_act_backward(g8, u8, h, recompute=True, stream=stream)
        out = [h, dg, du, again, q.act_read(c, stream=stream)]
        w, e = torch.zeros(96, 96, device=DEV), torch.zeros(50, 96, device=DEV)
        if stream is not None:
            stream.wait_stream(torch.cuda.current_stream())
        out.append(q.weight_grad(dg, c, w, stream=stream))
        out.append(q.embedding_lookup(tok, table, stream=stream))
        out.append(q.embedding_grad(tok, dg, e, stream=stream))
        return out

    want = run(None)
    torch.cuda.synchronize()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        torch.cuda._sleep(20_000_000)
        x.add_(0)
    got = run(side)
    side.synchronize()
    for a, b in zip(got, want):
        assert torch.equal(a, b)


def test_several_host_threads():
    want = {}
    blocks = {s: Block(seed=s, tokens=700 + 50 * s) for s in range(3)}
    for s, b in blocks.items():
        b.step()
        want[s] = [g.clone() for g in b.grads]
    torch.cuda.synchronize()
    bad = []

    def work(s):
        try:
            stream = torch.cuda.Stream()
            with torch.cuda.stream(stream):
                for _ in range(20):
                    for g in blocks[s].grads:
                        g.zero_()
                    blocks[s].step()
                    if not all(torch.equal(a, b) for a, b in zip(blocks[s].grads, want[s])):
                        bad.append(s)
            stream.synchronize()
        except Exception as e:      # noqa: BLE001  (reported below)
            bad.append(repr(e))

    threads = [threading.Thread(target=work, args=(s,)) for s in blocks]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not bad, bad


def test_past_four_gigabytes():
    """Rows whose byte offsets leave 32 bits, in every operand."""
    rows, pitch, n = 70_000, 65_536, 40
    x = torch.zeros(rows, pitch, dtype=B, device=DEV)
    gen = torch.Generator(device=DEV).manual_seed(1)
    part = torch.randint(-2, 3, (rows, n), generator=gen, device=DEV).to(B)
    cols = slice(pitch - n, pitch)
    x[:, cols] = part
    c = q.act_pack(x)
    assert c.data.numel() > 2 ** 32
    assert torch.equal(q.act_read(c)[:, cols], part)
    kept = c.data[-1000:, cols].clone()
    assert torch.equal(q.act_pack(part).data[-1000:, :n], kept)
    out = q.weight_grad(x[:, cols], part, torch.empty(n, n, device=DEV))
    exact = part.double().t() @ part.double()
    assert torch.equal(out.double(), exact)
    wide = q.weight_grad(part, c, torch.empty(n, pitch, device=DEV))
    assert torch.equal(wide[:, cols].double(), exact) and torch.all(wide[:, :pitch - n] == 0)
    h, g8, u8 = q.gated_act_forward(x[:, cols], x[:, cols])
    small = q.gated_act_forward(part, part)[0]
    assert torch.equal(h, small)
    del wide, c, g8, u8
    tok = torch.tensor([rows - 1, 0, rows - 1], device=DEV)
    assert torch.equal(q.embedding_lookup(tok, x)[:, cols], part[tok])
    x.zero_()
    q.embedding_grad(tok, torch.ones(3, n, device=DEV), x[:, cols], accumulate=True)
    assert x[rows - 1, -1] == 2 and x[0, -1] == 1 and x[:, cols].float().sum() == 3 * n
    say("large offsets: ok")


def test_refusals_on_the_gpu():
    x = torch.zeros(64, 64, dtype=B, device=DEV)
    _, g8, u8 = q.gated_act_forward(x, x.clone())
    for call in (lambda: q.gated_act_backward(g8, u8, x, dgate=x), lambda: q.gated_act_backward(g8, u8, x, dgate=x.clone()[:, :64], h=x),
                 lambda: q.gated_act_forward(x, x, gate_ckpt=g8, up_ckpt=g8),
                 lambda: q.weight_grad(x, x, x), lambda: q.embedding_lookup(torch.zeros(64, dtype=torch.int64, device=DEV), x, out=x),
                 lambda: q.embedding_grad(torch.zeros(64, dtype=torch.int64, device=DEV), x, x),
                 lambda: q.act_pack(x, q.ActCheckpoint(64, 64, data=x.view(torch.uint8).view(-1)[:4096].view(64, 64)))):
        with pytest.raises(q.QmuonError) as e:
            call()
        assert e.value.status == 1
    with pytest.raises(ValueError):
        q.act_pack(x, ckpt=q.ActCheckpoint(64, 64, device="cpu"))
    with pytest.raises(ValueError):
        q.weight_grad(x, x, torch.zeros(64, 64, device=DEV), ws=torch.zeros(10, 2, device=DEV)[:, 0])
