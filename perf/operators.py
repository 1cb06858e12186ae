"""The multi-tensor optimizer operators next to the Muon step, as cases to run and time.

AdamW with 32-bit states, AdamW with 8-bit states, the gradient's global norm
with its clip factor, and the three together as one training step uses them.
Each case runs the plain form (elementary torch operations) or, with `own`
set, the framework's entry points on the same buffers.

The tensors of a case are slices of flat buffers in which every tensor starts
on a 256-element boundary; what lies between two tensors is zero and stays
zero, so the plain form works on whole buffers, 256 elements to a row.
"""
import math

import torch

own = False

BLOCK = 256
LR, BETA1, BETA2, EPS, DECAY = 3e-4, 0.9, 0.999, 1e-8, 0.1
STEP = 1000          # mid-training: both bias corrections differ from 1
MAX_NORM, NORM_EPS = 0.25, 1e-6
TINY = 2.0 ** -100   # blocks of 8-bit states with a smaller maximum hold zeros
DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
SIZE = {"none": 0, "f32": 4, "bf16": 2, "f16": 2}


# ------------------------------------------------------------------ cases
# shapes8 / shapes32: "count x rows x cols, ..." of the tensors with 8-bit and
# 32-bit states (for op "clip": of the grads).  weight, grad, copy: types (the
# copy is the low-precision weight that the model computes with).  clip: the
# step takes its gradients times a clip factor.  pitch: columns of the fused
# buffer that the grads are column slices of (0: contiguous).  shift: elements
# by which the grads' buffer is off its allocation's alignment.

def _case(name, op, shapes8="", shapes32="", weight="f32", grad="f32", copy="none", rounding="nearest", clip=False,
          pitch=0, shift=0):
    c = dict(op=op, shapes8=shapes8, shapes32=shapes32, weight=weight, grad=grad, copy=copy, rounding=rounding,
             clip=clip, pitch=pitch, shift=shift)
    return dict(c, name=name) if name else c


def listed():
    layer = "2x4096x4096,2x1024x4096,2x14336x4096,1x4096x14336"
    return [
        # the norm gains of a 32-layer model: the smallest call, bound by its latency
        _case("adamw32_norms", "adamw", shapes32="65x1x4096"),
        # gains, biases and small odd matrices whose grads lie in a bucket at an odd offset
        _case("adamw32_odd", "adamw", shapes32="3x1x1,9x1x1000,2x17x129,12x333x1001", grad="bf16", shift=3),
        # one embedding kept in bf16
        _case("adamw32_embedding", "adamw", shapes32="1x50257x2048", weight="bf16", grad="bf16"),
        # a whole layer by AdamW: fp32 weights, the model's bf16 copy, clipped grads
        _case("adamw32_layer", "adamw", shapes32=layer, grad="bf16", copy="bf16", clip=True),
        # gains again, with 8-bit states
        _case("adamw8_norms", "adamw", shapes8="57x1x2048", weight="bf16", grad="bf16"),
        # stochastic codes, grads that are column slices of a fused buffer
        _case("adamw8_stochastic", "adamw", shapes8="2x6144x2048,2x2560x2048", weight="bf16", grad="bf16",
              rounding="stochastic", pitch=2304),
        # embedding and head: fp32 weights with the model's bf16 copy
        _case("adamw8_embeddings", "adamw", shapes8="2x50257x2048", grad="bf16", copy="bf16"),
        # a whole layer kept in bf16
        _case("adamw8_layer", "adamw", shapes8=layer, weight="bf16", grad="bf16"),
        # clipping the grads of the norm gains
        _case("clip_norms", "clip", shapes32="65x1x4096"),
        # fp16 grads inside a fused buffer
        _case("clip_slices", "clip", shapes32="4x6144x2048,1x2560x2048", grad="f16", pitch=2304),
        # every grad of a 28-layer model
        _case("clip_model", "clip", shapes32="28x2560x2048,28x2048x2048,56x6144x2048,28x2048x6144", grad="bf16"),
        # what a Muon program leaves to AdamW, in one step: norm of all grads, 8-bit embedding and head, 32-bit gains
        _case("step_embeddings_norms", "adamw", shapes8="2x32000x4096", shapes32="65x1x4096", grad="bf16", copy="bf16",
              clip=True),
    ]


def draw(rng):
    def count(lo, hi):
        return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))

    def shapes(total, pitch):
        groups, left = [], total
        for _ in range(rng.randint(1, 3)):
            cols = 256 * rng.randint(1, 16) if pitch else count(1, min(9000, left))
            n = count(1, max(1, min(40, left // cols)))
            rows = 1 if not pitch and rng.random() < 0.3 else max(1, left // (cols * n))
            if pitch and groups:
                break
            groups.append("%dx%dx%d" % (n, rows, cols))
            left = max(left - n * rows * cols, 256)
        return ",".join(groups)

    op = rng.choice(["adamw", "adamw", "adamw", "clip"])
    pitched = rng.random() < 0.25
    total = count(1000, 4.0e8 if op == "clip" else 1.0e8)
    kind = rng.choice(["8", "32"] if pitched else ["8", "32", "both"])
    s = shapes(total, pitched)
    pitch = int(s.split("x")[-1]) + 8 * rng.randint(1, 40) if pitched else 0
    grad, shift = rng.choice(["f32", "bf16", "bf16", "f16"]), 0 if pitched else rng.choice([0, 0, 1, 4])
    if op == "clip":
        return _case(None, op, shapes32=s, grad=grad, pitch=pitch, shift=shift)
    weight = rng.choice(["f32", "f32", "bf16", "f16"])
    return _case(None, op, shapes8=s if kind != "32" else "",
                 shapes32=s if kind == "32" else shapes(count(300, 3e5), False) if kind == "both" else "",
                 weight=weight, grad=grad, copy=rng.choice(["none", "bf16", "f16"]) if weight == "f32" else "none",
                 rounding=rng.choice(["nearest", "stochastic"]) if kind != "32" else "nearest",
                 clip=rng.random() < 0.5, pitch=pitch, shift=shift)


# ----------------------------------------------------------------- inputs

def _shapes(text):
    out = []
    for part in filter(None, text.split(",")):
        n, rows, cols = (int(v) for v in part.split("x"))
        out += [(rows, cols)] * n
    return out


def _blocks(rows, cols):
    return -(-rows * cols // BLOCK)


class _Group:
    """The tensors of one kind of state, as slices of flat buffers."""


def _group(case, bits, shapes, seed, first_tensor):
    dev = "cuda"
    gen = torch.Generator(device=dev)
    gen.manual_seed(1000003 * seed + bits)
    G = _Group()
    G.bits, G.shapes = bits, shapes
    nbs = [_blocks(r, c) for r, c in shapes]
    G.nb = sum(nbs)
    n = G.nb * BLOCK
    count = torch.tensor(nbs, device=dev)
    start = torch.cumsum(count, 0) - count
    G.tensor = torch.repeat_interleave(torch.arange(len(shapes), device=dev), count)      # tensor of each block
    G.block = torch.arange(G.nb, device=dev) - start[G.tensor]                             # its index in the tensor
    G.tensor = G.tensor + first_tensor                                                     # index in the step's list
    G.at = [int(v) * BLOCK for v in start.tolist()]
    # matrices decay, vectors do not; every third tensor has half the step size
    G.decays = [DECAY if r > 1 else 0.0 for r, c in shapes]
    G.scales = [0.5 if (first_tensor + i) % 3 == 2 else 1.0 for i in range(len(shapes))]
    G.decay = torch.repeat_interleave(torch.tensor(G.decays, device=dev), count)[:, None]
    G.scale = torch.repeat_interleave(torch.tensor(G.scales, device=dev), count)[:, None]

    def normal(*shape):
        return torch.randn(*shape, generator=gen, device=dev)

    def uniform(*shape):
        return torch.rand(*shape, generator=gen, device=dev)

    left = torch.tensor([r * c for r, c in shapes], device=dev)[G.tensor - first_tensor] - G.block * BLOCK
    inside = (torch.arange(BLOCK, device=dev)[None, :] < left[:, None]) if any(r * c % BLOCK for r, c in shapes) else None
    # grads of every block's own size, an eighth of the blocks untouched so far (rows of an embedding)
    sigma = 1e-3 * torch.exp(0.7 * normal(G.nb, 1)) * (uniform(G.nb, 1) > 0.125)

    def masked(x):
        return x if inside is None else x * inside

    g = masked(normal(G.nb, BLOCK) * sigma).to(DTYPES[case["grad"]])
    if case["pitch"]:
        rows, cols = sum(r for r, c in shapes), shapes[0][1]
        G.buffer = torch.zeros(rows, case["pitch"], dtype=g.dtype, device=dev)
        G.buffer[:, :cols] = g.view(rows, cols)
        G.g = G.buffer[:, :cols]
    else:
        G.buffer = torch.zeros(n + 8, dtype=g.dtype, device=dev)
        G.g = G.buffer[case["shift"]:case["shift"] + n]
        G.g.copy_(g.view(-1))
    del g
    if case["op"] == "clip":
        return G
    G.w = masked(normal(G.nb, BLOCK) * 0.02).to(DTYPES[case["weight"]]).view(-1)
    G.copy = torch.zeros(n, dtype=DTYPES[case["copy"]], device=dev) if case["copy"] != "none" else None
    if bits == 32:
        G.m = masked(normal(G.nb, BLOCK) * (0.25 * sigma)).view(-1)
        G.v = masked((0.5 + uniform(G.nb, BLOCK)) * (sigma * sigma)).view(-1)
    else:
        alive = sigma > 0
        G.m = masked((normal(G.nb, BLOCK) * 36).round().clamp(-127, 127) * alive).to(torch.int8).view(-1)
        G.m_absmax = (0.7 * sigma * (0.5 + uniform(G.nb, 1))).view(-1)
        G.v = masked((180 + 25 * normal(G.nb, BLOCK)).round().clamp(1, 255) * alive).to(torch.uint8).view(-1)
        G.v_absmax = (2 * sigma * sigma * (0.5 + uniform(G.nb, 1))).view(-1)
    return G


class _State:
    pass


def _inputs(case, seed):
    S = _State()
    S.case, S.seed = case, seed
    S.groups = []
    tensors = 0
    for bits in (8, 32):
        shapes = _shapes(case["shapes%d" % bits])
        if shapes:
            S.groups.append(_group(case, bits, shapes, seed, tensors))
            tensors += len(shapes)
    return S


def _slices(G, flat):
    return [flat[a:a + r * c] for a, (r, c) in zip(G.at, G.shapes)]


def _grads(G, case):
    if not case["pitch"]:
        return _slices(G, G.g)
    out, row = [], 0
    for r, c in G.shapes:
        out.append(G.g[row:row + r])
        row += r
    return out


def prepare(case, seed):
    S = _inputs(case, seed)
    if own:
        import quantized_momentum_newton_amd as q
        if case["clip"] or case["op"] == "clip":
            S.grads = q.GradPlan([g for G in S.groups for g in _grads(G, case)])
            S.ws = S.grads.workspace()
        if case["op"] == "adamw":
            tensors = []
            for G in S.groups:
                w, g = _slices(G, G.w), _grads(G, case)
                m, v = _slices(G, G.m), _slices(G, G.v)
                copy = _slices(G, G.copy) if G.copy is not None else [None] * len(w)
                for i in range(len(w)):
                    n = w[i].numel()
                    scales = {}
                    if G.bits == 8:
                        b = slice(G.at[i] // BLOCK, G.at[i] // BLOCK + -(-n // BLOCK))
                        scales = dict(m_absmax=G.m_absmax[b], v_absmax=G.v_absmax[b])
                    state = q.AdamWState(n, bits=G.bits, m=m[i], v=v[i], **scales)
                    tensors.append((w[i], g[i], state, copy[i], G.scales[i], G.decays[i]))
            S.plan = q.AdamWPlan(tensors)
    return S


# -------------------------------------------------------------- one pass

def run(S):
    return _run_own(S) if own else _run_plain(S)


def _answer(S, norm, coef, states):
    out = {}
    if norm is not None:
        out["norm"], out["coef"] = norm, coef
    if S.case["op"] == "clip":
        out["grads"] = [G.g for G in S.groups]
        return out
    out["weight"] = [G.w for G in S.groups]
    if S.case["copy"] != "none":
        out["copy"] = [G.copy for G in S.groups]
    out["m"], out["v"] = [m for m, _ in states], [v for _, v in states]
    return out


def _run_own(S):
    import quantized_momentum_newton_amd as q
    case = S.case
    norm = coef = None
    if case["clip"] or case["op"] == "clip":
        norm, coef = q.grad_norm(S.grads, MAX_NORM, eps=NORM_EPS, ws=S.ws)
    if case["op"] == "clip":
        q.grad_scale(S.grads, coef)
        return _answer(S, norm, coef, None)
    q.adamw_step(S.plan, STEP, lr=LR, betas=(BETA1, BETA2), eps=EPS, grad_scale=coef, rounding=case["rounding"],
                 seed=S.seed)
    if S.groups[0].bits == 32:
        return _answer(S, norm, coef, [(G.m, G.v) for G in S.groups])
    # 8-bit states leave as the values they stand for, block after block
    m, v = q.adamw_read_state(S.plan)
    states, at = [], 0
    for G in S.groups:
        n = G.nb * BLOCK
        states.append((m[at:at + n], v[at:at + n]))
        at += n
    return _answer(S, norm, coef, states)


def _run_plain(S):
    case = S.case
    norm = coef = None
    if case["clip"] or case["op"] == "clip":
        total = sum(G.g.double().square().sum() for G in S.groups)
        root = total.sqrt()
        norm, coef = root.float().view(1), (MAX_NORM / (root + NORM_EPS)).clamp(max=1.0).float().view(1)
    if case["op"] == "clip":
        for G in S.groups:
            G.g.copy_(G.g.float() * coef)
        return _answer(S, norm, coef, None)
    return _answer(S, norm, coef, [_plain_step(S, G, coef) for G in S.groups])


def _plain_step(S, G, coef):
    g = G.g.reshape(G.nb, BLOCK).float()
    if coef is not None:
        g = g * coef
    if G.bits == 32:
        m = G.m.view(G.nb, BLOCK) * BETA1 + g * (1 - BETA1)
        v = G.v.view(G.nb, BLOCK) * BETA2 + (g * g) * (1 - BETA2)
    else:
        # binary32 in this order, so that the codes are the same wherever they are computed
        step_m = (G.m_absmax / torch.full_like(G.m_absmax, 127.0)) * BETA1
        step_v = (G.v_absmax / torch.full_like(G.v_absmax, 65025.0)) * BETA2
        c = G.v.view(G.nb, BLOCK).float()
        m = G.m.view(G.nb, BLOCK).float() * step_m[:, None] + g * (1 - BETA1)
        v = (c * c) * step_v[:, None] + (g * g) * (1 - BETA2)
    lr = LR * G.scale
    w = G.w.view(G.nb, BLOCK).float()
    denom = v.sqrt() * (1 / math.sqrt(1 - BETA2 ** STEP)) + EPS
    w = w - w * (lr * G.decay) - (m / denom) * (lr / (1 - BETA1 ** STEP))
    G.w.copy_(w.view(-1))
    if G.copy is not None:
        G.copy.copy_(w.view(-1))
    if G.bits == 32:
        G.m.copy_(m.view(-1))
        G.v.copy_(v.view(-1))
        return G.m, G.v
    return _plain_requantise(S, G, m, v)


def _plain_requantise(S, G, m, v):
    one = torch.ones_like(G.m_absmax)
    top_m, top_v = m.abs().amax(1), v.amax(1)
    top_m, top_v = torch.where(top_m < TINY, 0.0, top_m), torch.where(top_v < TINY, 0.0, top_v)
    inv_m = torch.where(top_m > 0, (one * 127.0) / top_m, 0.0)
    inv_v = torch.where(top_v > 0, (one * 65025.0) / top_v, 0.0)
    x, y = m * inv_m[:, None], v * inv_v[:, None]
    # next to a border: the root and its square in 64 bits
    k = y.double().sqrt().floor()
    above = y.double() - k * k
    if S.case["rounding"] == "nearest":
        code_m = x.round()
        up = above > k + 0.5
    else:
        word = _words(G, S.seed)
        code_m = x.floor()
        code_m = code_m + (word.bitwise_right_shift(16).float() * 2.0 ** -16 < x - code_m)
        up = above > (word.bitwise_and(0x7FFF).double() * 2.0 ** -15) * (2 * k + 1)
    code_v = torch.where((v > 0) & (top_v > 0)[:, None], (k + up).clamp(1, 255), 0.0)
    G.m.copy_(code_m.clamp(-127, 127).view(-1))
    G.v.copy_(code_v.view(-1))
    G.m_absmax.copy_(top_m)
    G.v_absmax.copy_(top_v)
    c = G.v.view(G.nb, BLOCK).float()
    m = G.m.view(G.nb, BLOCK).float() * (top_m / (one * 127.0))[:, None]
    v = (c * c) * (top_v / (one * 65025.0))[:, None]
    return m.view(-1), v.view(-1)


def _words(G, seed):
    """The 32-bit random number of every element: Philox4x32-10 with the
    counter (element / 4, step, tensor) and the seed as its key."""
    quad = torch.arange(BLOCK // 4, device=G.block.device)[None, :] + G.block[:, None] * (BLOCK // 4)
    low = 0xFFFFFFFF
    c0, c1 = quad & low, quad >> 32
    c2, c3 = torch.full_like(quad, STEP), G.tensor[:, None].expand_as(quad)
    k0, k1 = seed & low, seed >> 32
    for _ in range(10):
        # products modulo 2^64: their upper and lower halves
        p0, p1 = c0 * 0xD2511F53, c2 * 0xCD9E8D57
        c0, c1, c2, c3 = ((p1 >> 32) & low) ^ c1 ^ k0, p1 & low, ((p0 >> 32) & low) ^ c3 ^ k1, p0 & low
        k0, k1 = (k0 + 0x9E3779B9) & low, (k1 + 0xBB67AE85) & low
    return torch.stack((c0, c1, c2, c3), dim=2).view(G.nb, BLOCK)


# ------------------------------------------------------------------ bounds

def work(case):
    """Grads read (and written back by a clip), weights, states and scales read
    and written, copies and the values of 8-bit states written, once each."""
    bytes_, flops = 0, 0
    for bits in (8, 32):
        n = sum(r * c for r, c in _shapes(case["shapes%d" % bits]))
        nb = sum(_blocks(r, c) for r, c in _shapes(case["shapes%d" % bits]))
        if case["op"] == "clip":
            bytes_ += n * 2 * SIZE[case["grad"]]
            flops += 3 * n
        else:
            state = 16 * n if bits == 32 else 4 * n + 16 * nb + 8 * n
            bytes_ += n * (SIZE[case["grad"]] + 2 * SIZE[case["weight"]] + SIZE[case["copy"]]) + state
            flops += n * ((15 if bits == 32 else 26) + (3 if case["clip"] else 0))
    return {"bytes": bytes_, "flops": flops}


# ----------------------------------------------------------- in 64 bits

def exact(case, seed):
    """Weights, norms and 32-bit states in 64 bits throughout.  The codes of
    8-bit states are defined by binary32 operations in a stated order: each
    operation is done in 64 bits here and rounded to 32 where the definition
    rounds (exact for sums, products, quotients of 32-bit numbers)."""
    S = _inputs(case, seed)
    grads = [G.g.double() for G in S.groups]
    norm = coef = factor = None
    if case["clip"] or case["op"] == "clip":
        norm = torch.linalg.vector_norm(torch.stack([torch.linalg.vector_norm(g) for g in grads]))
        factor = min(1.0, MAX_NORM / (float(norm) + NORM_EPS))
        norm, coef = norm.view(1), torch.tensor([factor], dtype=torch.float64)
    if case["op"] == "clip":
        return {"norm": norm, "coef": coef, "grads": [g * factor for g in grads]}
    out = {"weight": [], "m": [], "v": []}
    for G, g in zip(S.groups, grads):
        g = g.reshape(-1, BLOCK)
        scaled = g if factor is None else g * factor
        if G.bits == 32:
            m0, v0 = G.m.double().view(-1, BLOCK), G.v.double().view(-1, BLOCK)
        else:
            m0 = G.m.double().view(-1, BLOCK) * (G.m_absmax.double() / 127)[:, None]
            v0 = G.v.double().view(-1, BLOCK).square() * (G.v_absmax.double() / 65025)[:, None]
        m, v = BETA1 * m0 + (1 - BETA1) * scaled, BETA2 * v0 + (1 - BETA2) * scaled.square()
        lr = LR * G.scale.double()
        hat = (m / (1 - BETA1 ** STEP)) / ((v / (1 - BETA2 ** STEP)).sqrt() + EPS)
        w = G.w.double().view(-1, BLOCK)
        out["weight"].append((w * (1 - lr * G.decay.double()) - lr * hat).view(-1))
        del m0, v0, hat, w
        if G.bits == 8:
            m, v = _exact_states(S, G, g, factor)
        out["m"].append(m.view(-1))
        out["v"].append(v.view(-1))
    if case["copy"] != "none":
        out["copy"] = out["weight"]
    if norm is not None:
        out["norm"], out["coef"] = norm, coef
    return out


def _r32(x):
    return x.float().double()


def _exact_states(S, G, g, factor):
    def const(v):
        return float(torch.tensor(v, dtype=torch.float64).float())

    b1, a1, b2, a2 = const(BETA1), const(1 - BETA1), const(BETA2), const(1 - BETA2)
    if factor is not None:
        g = _r32(g * const(factor))
    sm, sv = _r32(_r32(G.m_absmax.double() / 127) * b1), _r32(_r32(G.v_absmax.double() / 65025) * b2)
    m = _r32(_r32(G.m.view(-1, BLOCK).double() * sm[:, None]) + _r32(g * a1))
    v = _r32(_r32(G.v.view(-1, BLOCK).double().square() * sv[:, None]) + _r32(_r32(g * g) * a2))
    del g
    top_m, top_v = m.abs().max(1, keepdim=True).values, v.max(1, keepdim=True).values
    top_m[top_m < TINY] = 0
    top_v[top_v < TINY] = 0
    x = _r32(m * torch.nan_to_num(_r32(127 / top_m), posinf=0.0))
    y = _r32(v * torch.nan_to_num(_r32(65025 / top_v), posinf=0.0))
    positive = (v > 0) & (top_v > 0)
    del m, v
    base = torch.floor(torch.sqrt(y))
    if S.case["rounding"] == "nearest":
        codes, threshold = torch.round(x), 0.5
    else:
        word = _words(G, S.seed)
        down = torch.floor(x)
        codes = torch.where((word >> 16).double() / 65536 < x - down, down + 1, down)
        threshold = (word & 32767).double() / 32768
    roots = torch.where(y - base ** 2 > threshold * ((base + 1) ** 2 - base ** 2), base + 1, base)
    roots = torch.where(positive, roots.clamp(1, 255), torch.zeros_like(roots))
    return codes.clamp(-127, 127) * (top_m / 127), roots.square() * (top_v / 65025)
