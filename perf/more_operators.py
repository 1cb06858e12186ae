"""The operators that make the gradients an optimizer step reads, as cases to
run and time.

Activations kept in 8 bits for the backward pass, the weight gradient that is
formed from them, the gated activation that writes and reads them, and the
embedding lookup with its gradient.  Each case runs the plain form (elementary
torch operations) or, with `own` set, the framework's entry points on the same
buffers.
"""
import math

import torch

own = False

GROUP = 32           # rows of a column that share a scale
E4M3_MAX = 448.0
LOW, HIGH = -95, 119  # exponents a scale can have
DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
SIZE = {"f32": 4, "bf16": 2, "f16": 2}
GELU = math.sqrt(2 / math.pi)


# ------------------------------------------------------------------ cases
# pitch: row pitch in elements of the inputs that are column slices of a wider
# buffer (0: contiguous).

def _checkpoint(rows, cols, kind, pitch=0):
    return dict(op="checkpoint", rows=rows, cols=cols, kind=kind, pitch=pitch)


def _weight(rows, n, k, kind="bf16", kept=True, out="f32", accumulate=True, pitch=0):
    return dict(op="weight_grad", rows=rows, n=n, k=k, kind=kind, kept=kept, out=out, accumulate=accumulate, pitch=pitch)


def _gated(rows, cols, kind="bf16", act="silu", fused=True):
    return dict(op="gated", rows=rows, cols=cols, kind=kind, act=act, fused=fused)


def _embedding(tokens, vocab, cols, table="f32", kind="bf16", grad="f32", accumulate=False, padded=False):
    return dict(op="embedding", tokens=tokens, vocab=vocab, cols=cols, table=table, kind=kind, grad=grad,
                accumulate=accumulate, padded=padded)


def listed():
    return [
        # a short sequence of odd width: two launches, bound by their latency
        dict(_checkpoint(40, 1001, "bf16"), name="checkpoint_short"),
        # the input of a layer's projections
        dict(_checkpoint(8192, 4096, "bf16"), name="checkpoint_layer"),
        # one matrix of a small model, added to its gradient buffer
        dict(_weight(1024, 512, 256), name="weight_grad_small"),
        # the widest projection of a layer
        dict(_weight(8192, 14336, 4096), name="weight_grad_layer"),
        # many tokens and a narrow product, operands not packed
        dict(_weight(65536, 1024, 2048, "f16", kept=False, accumulate=False), name="weight_grad_long"),
        # odd sizes, dy a slice of a fused buffer, bf16 gradients
        dict(_weight(5001, 2047, 1001, kept=False, out="bf16", pitch=2304), name="weight_grad_odd"),
        # a small model's feed-forward block
        dict(_gated(100, 512), name="gated_small"),
        # gate and up from one fused projection
        dict(_gated(8192, 14336), name="gated_layer"),
        # the tanh form of gelu, separate projections of odd width, f16
        dict(_gated(3001, 6145, "f16", "gelu", fused=False), name="gated_odd"),
        # a small model's table in fp32
        dict(_embedding(1024, 512, 256, kind="f32"), name="embedding_small"),
        # a large vocabulary, the gradient table written whole
        dict(_embedding(32768, 50257, 2048), name="embedding_vocabulary"),
        # a bf16 table tied to the head: added to the head's gradient, ragged sequences padded with -1
        dict(_embedding(16384, 32000, 4096, "bf16", "bf16", "bf16", accumulate=True, padded=True), name="embedding_tied"),
    ]


def draw(rng):
    def size(lo, hi):
        return max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi))))))

    def width(lo, hi):
        n = size(lo, hi)
        return n if rng.random() < 0.4 else max(lo, n // 64 * 64)

    op = rng.choice(["checkpoint", "weight_grad", "weight_grad", "gated", "embedding"])
    if op == "checkpoint":
        cols = width(64, 16384)
        rows = size(1, min(65536, 3.3e7 / cols))
        return _checkpoint(rows, cols, rng.choice(["f32", "bf16", "f16"]), rng.choice([0, 0, cols + rng.randint(1, 200)]))
    if op == "weight_grad":
        n, k = width(32, 14336), width(32, 8192)
        rows = size(1, max(2, min(65536, 4.8e11 / n / k, 2.7e8 / max(n, k))))
        return _weight(rows, n, k, rng.choice(["bf16", "bf16", "f16"]), rng.random() < 0.6, rng.choice(["f32", "f32", "bf16"]),
                       rng.random() < 0.6, rng.choice([0, 0, n + 8 * rng.randint(1, 40)]))
    if op == "gated":
        cols = width(64, 16384)
        return _gated(size(1, min(65536, 1.1e8 / cols)), cols, rng.choice(["bf16", "bf16", "f16", "f32"]),
                      rng.choice(["silu", "gelu"]), rng.random() < 0.6)
    cols, vocab = width(32, 8192), size(100, 130000)
    vocab = min(vocab, int(1.3e8 / cols))
    return _embedding(size(1, min(131072, 1e8 / cols)), vocab, cols, rng.choice(["f32", "bf16"]), rng.choice(["f32", "bf16", "f16"]),
                      rng.choice(["f32", "bf16"]), rng.random() < 0.5, rng.random() < 0.3)


# ----------------------------------------------------------------- inputs

class _State:
    pass


def _normal(gen, *shape):
    return torch.randn(*shape, generator=gen, device="cuda")


def _activations(gen, rows, cols):
    """Columns of their own sizes, one in 64 an outlier."""
    size = torch.exp(0.5 * _normal(gen, cols)) * torch.where(torch.rand(cols, generator=gen, device="cuda") < 1 / 64, 20.0, 1.0)
    return _normal(gen, rows, cols) * size


def _pitched(x, pitch, dtype):
    if not pitch:
        return x.to(dtype)
    wide = torch.zeros(x.shape[0], pitch, dtype=dtype, device="cuda")
    wide[:, :x.shape[1]] = x
    return wide[:, :x.shape[1]]


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    S = _State()
    S.case, kind = case, DTYPES[case.get("kind", "f32")]
    if case["op"] == "checkpoint":
        S.x = _pitched(_activations(gen, case["rows"], case["cols"]), case["pitch"], kind)
    elif case["op"] == "weight_grad":
        rows, n, k = case["rows"], case["n"], case["k"]
        S.dy = _pitched(1e-2 * _normal(gen, rows, n), case["pitch"], kind)
        x = _activations(gen, rows, k)
        if case["kept"]:      # kept by the forward pass: bytes and scales in rows of a multiple of 16
            codes, e = _codes(x)
            S.data, S.scale = (torch.zeros(len(v), -(-k // 16) * 16, dtype=torch.uint8, device="cuda") for v in (x, e))
            S.data[:, :k] = codes.view(torch.uint8)
            S.scale[:, :k] = (e + 127).to(torch.uint8)
        else:
            S.x = x.to(kind)
        S.out = (_normal(gen, n, k) * 1e-2 * math.sqrt(rows)).to(DTYPES[case["out"]])
        if own:
            import quantized_momentum_newton_amd as q
            if case["kept"]:
                S.x = q.ActCheckpoint(rows, k, data=S.data, scale=S.scale)
            S.ws = q.weight_grad_workspace(S.dy, S.x, S.out)
    elif case["op"] == "gated":
        rows, cols = case["rows"], case["cols"]
        wide = torch.cat([2 * _normal(gen, rows, cols), _activations(gen, rows, cols)], 1).to(kind)
        if case["fused"]:
            S.gate, S.up = wide[:, :cols], wide[:, cols:]
            S.grads = torch.zeros_like(wide)
            S.dgate, S.dup = S.grads[:, :cols], S.grads[:, cols:]
        else:
            S.gate, S.up = wide[:, :cols].clone(), wide[:, cols:].clone()
            S.dgate, S.dup = torch.zeros_like(S.gate), torch.zeros_like(S.up)
        S.dh = (1e-2 * _normal(gen, rows, cols)).to(kind)
    else:
        tokens, vocab, cols = case["tokens"], case["vocab"], case["cols"]
        # frequencies as one over the rank, ranks spread over the vocabulary
        rank = torch.exp(torch.rand(tokens, generator=gen, device="cuda") * math.log(vocab)).long() - 1
        S.tokens = torch.randperm(vocab, generator=gen, device="cuda")[rank.clamp(0, vocab - 1)]
        if case["padded"]:
            S.tokens[torch.rand(tokens, generator=gen, device="cuda") < 0.1] = -1
        S.table = (0.02 * _normal(gen, vocab, cols)).to(DTYPES[case["table"]])
        S.dy = (1e-2 * _normal(gen, tokens, cols)).to(kind)
        S.grad = (1e-2 * _normal(gen, vocab, cols)).to(DTYPES[case["grad"]])
        if own:
            import quantized_momentum_newton_amd as q
            S.ws = q.embedding_grad_workspace(S.tokens, S.dy, S.grad)
    return S


# -------------------------------------------------------------- one pass

def run(S):
    return _run_own(S) if own else _run_plain(S)


def _run_own(S):
    import quantized_momentum_newton_amd as q
    case = S.case
    if case["op"] == "checkpoint":
        return q.act_read(q.act_pack(S.x), dtype=S.x.dtype)
    if case["op"] == "weight_grad":
        q.weight_grad(S.dy, S.x, S.out, accumulate=case["accumulate"], ws=S.ws)
        return S.out
    if case["op"] == "gated":
        h, gate, up = q.gated_act_forward(S.gate, S.up, act=case["act"])
        _, _, again = q.gated_act_backward(gate, up, S.dh, S.dgate, S.dup, recompute=True, act=case["act"])
        return {"h": h, "again": again, "grads": S.grads if case["fused"] else [S.dgate, S.dup]}
    scale = math.sqrt(case["cols"])
    out = q.embedding_lookup(S.tokens, S.table, scale, dtype=S.dy.dtype)
    q.embedding_grad(S.tokens, S.dy, S.grad, scale, accumulate=case["accumulate"], ws=S.ws)
    return {"out": out, "grad": S.grad}


def _run_plain(S):
    case = S.case
    if case["op"] == "checkpoint":
        return _values(*_codes(S.x)).to(S.x.dtype)
    if case["op"] == "weight_grad":
        if case["kept"]:
            k = case["k"]
            x = _values(S.data[:, :k].view(torch.float8_e4m3fn), S.scale[:, :k].int() - 127)
            x = x.to(S.dy.dtype).float()      # the product's operands have dy's type
        else:
            x = S.x.float()
        d = S.dy.float().t() @ x
        S.out.copy_(S.out.float() + d if case["accumulate"] else d)
        return S.out
    if case["op"] == "gated":
        h = (_act(S.gate.float(), case["act"])[0] * S.up.float()).to(S.dh.dtype)
        gate, up = _values(*_codes(S.gate)), _values(*_codes(S.up))
        a, slope = _act(gate, case["act"])
        dh = S.dh.float()
        S.dgate.copy_(dh * up * slope)
        S.dup.copy_(dh * a)
        return {"h": h, "again": (a * up).to(S.dh.dtype), "grads": S.grads if case["fused"] else [S.dgate, S.dup]}
    scale = math.sqrt(case["cols"])
    inside = (S.tokens >= 0)[:, None]
    at = S.tokens.clamp(min=0)
    out = (S.table[at].float() * (inside * scale)).to(S.dy.dtype)
    d = torch.zeros(S.grad.shape, device="cuda").index_add_(0, at, S.dy.float() * inside) * scale
    S.grad.copy_(S.grad.float() + d if case["accumulate"] else d)
    return {"out": out, "grad": S.grad}


def _codes(x):
    """E4M3 numbers of x over a power of two, and its exponent, one for 32 rows of a column."""
    rows, cols = x.shape
    groups = -(-rows // GROUP)
    x = torch.nn.functional.pad(x.float(), (0, 0, 0, groups * GROUP - rows)).view(groups, GROUP, cols)
    # the smallest power of two that brings the largest to at most 448 = 1.75 * 2^8
    e = ((x.abs().amax(1).view(torch.int32) + 0x1FFFFF >> 23) - 135).clamp(LOW, HIGH)
    y = x * (127 - e << 23).view(torch.float32)[:, None]
    return y.clamp(-E4M3_MAX, E4M3_MAX).to(torch.float8_e4m3fn).view(groups * GROUP, cols)[:rows], e


def _values(codes, e):
    unit = (e + 127 << 23).view(torch.float32)
    return codes.float() * unit.repeat_interleave(GROUP, 0)[:len(codes)]


def _act(x, act):
    """The activation and its derivative."""
    if act == "silu":
        s = 1 / (1 + torch.exp(-x))
        return x * s, s * (1 + x * (1 - s))
    s = 1 / (1 + torch.exp(-2 * GELU * (x + 0.044715 * x * x * x)))
    return x * s, s + x * (s * (1 - s)) * (2 * GELU * (1 + 3 * 0.044715 * x * x))


# ------------------------------------------------------------------ bounds

def work(case):
    """Inputs read and outputs written once each; what is kept in 8 bits has a
    byte an element and a scale for 32 of them."""
    kept = 33 / 32
    if case["op"] == "checkpoint":
        n = case["rows"] * case["cols"]
        return {"bytes": n * (2 * SIZE[case["kind"]] + 2 * kept), "flops": 4 * n}
    if case["op"] == "weight_grad":
        t, n, k = case["rows"], case["n"], case["k"]
        x = kept if case["kept"] else SIZE[case["kind"]]
        return {"bytes": t * n * SIZE[case["kind"]] + t * k * x + n * k * SIZE[case["out"]] * (1 + case["accumulate"]),
                "flops": 2 * t * n * k}
    if case["op"] == "gated":
        n = case["rows"] * case["cols"]
        return {"bytes": n * (7 * SIZE[case["kind"]] + 4 * kept), "flops": 40 * n}
    n, rows = case["tokens"] * case["cols"], min(case["tokens"], case["vocab"]) * case["cols"]
    table = 2 * rows if case["accumulate"] else case["vocab"] * case["cols"]
    return {"bytes": case["tokens"] * 8 + rows * SIZE[case["table"]] + 2 * n * SIZE[case["kind"]] + table * SIZE[case["grad"]],
            "flops": 3 * n}


# ----------------------------------------------------------- in 64 bits

def exact(case, seed):
    S = prepare(case, seed)
    if case["op"] == "checkpoint":
        return _kept64(S.x.double())
    if case["op"] == "weight_grad":
        if case["kept"]:
            x = _decode64(S.data[:, :case["k"]], S.scale[:, :case["k"]])
            x = x.to(S.dy.dtype).double() if case["kind"] == "f16" else x
        else:
            x = S.x.double()
        d = torch.matmul(S.dy.double().t(), x)
        return d + S.out.double() if case["accumulate"] else d
    if case["op"] == "gated":
        h = _act64(S.gate.double(), case["act"])[0].mul_(S.up.double())
        up = _kept64(S.up.double())
        a, slope = _act64(_kept64(S.gate.double()), case["act"])
        dh = S.dh.double()
        grads = [dh * up * slope, dh * a]
        return {"h": h, "again": a * up, "grads": torch.cat(grads, 1) if case["fused"] else grads}
    scale, real = math.sqrt(case["cols"]), S.tokens >= 0
    out = torch.zeros(len(S.tokens), case["cols"], dtype=torch.float64, device="cuda")
    out[real] = S.table[S.tokens[real]].double() * scale
    grad = S.grad.double() if case["accumulate"] else torch.zeros(S.grad.shape, dtype=torch.float64, device="cuda")
    grad.index_put_((S.tokens[real],), S.dy[real].double() * scale, accumulate=True)
    return {"out": out, "grad": grad}


def _kept64(x):
    """x as its 8 bits hold it: in each column's 32 rows a common unit 2^e, e
    the smallest integer with |x| <= 448 * 2^e, and multiples of 2^(k-3) of it
    for numbers of 2^k to 2^(k+1), of 2^-9 below 2^-6."""
    out = torch.empty_like(x)
    groups = x.shape[0] // GROUP
    for rows in (slice(0, groups * GROUP), slice(groups * GROUP, None)):
        part = x[rows]
        if part.numel():
            part = part.reshape(max(1, groups if rows.start == 0 else 1), -1, x.shape[1])
            top = part.abs().max(1, keepdim=True).values
            frac, power = torch.frexp(top / E4M3_MAX)          # frac in [1/2, 1)
            e = torch.where(top > 0, torch.where(frac > 0.5, power, power - 1), LOW).clamp(LOW, HIGH)
            y = (part * _two(-e)).clamp(-E4M3_MAX, E4M3_MAX)
            step = torch.frexp(y).exponent.sub(1).clamp(min=-6) - 3
            out[rows] = ((y * _two(-step)).round() * _two(step + e)).reshape(-1, x.shape[1])
    return out


def _two(e):
    """2^e, its bits put together."""
    return (e.long() + 1023 << 52).view(torch.float64)


def _decode64(data, scale):
    b = data.double()
    sign = torch.where(b >= 128, -1.0, 1.0)
    b = torch.where(b >= 128, b - 128, b)
    power, m = torch.floor(b / 8), torch.remainder(b, 8)
    y = sign * torch.where(power > 0, (1 + m / 8) * _two(power - 7), m * 2.0 ** -9)
    rows = torch.arange(len(b), device="cuda") // GROUP
    return y * _two(scale.long() - 127)[rows]


def _act64(x, act):
    if act == "silu":
        s = torch.sigmoid(x)
        return x * s, s + x * s * torch.sigmoid(-x)
    z = GELU * (x + 0.044715 * x ** 3)
    t = torch.tanh(z)
    return 0.5 * x * (1 + t), 0.5 * (1 + t) + 0.5 * x * (1 - t ** 2) * GELU * (1 + 3 * 0.044715 * x ** 2)
