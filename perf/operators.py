"""What is measured of the layer products with an epilogue, their expert-grouped
form, and the AdamW step: the cases, their inputs, their plain forms in
elementary torch operations, and the calls a user makes (``own``).

Operators
  epilogue  Y = act(X @ W^T + bias) + residual, W[n, k] = q[n, k] * s[n] held as
            int6 / int8 codes in the tile layout of ``gq.tile_weight``
  grouped   the same product for rows sorted by expert, with ragged counts
  adamw     one AdamW step over a list of tensors, states in 32 or in 8 bits
"""
import math

import numpy as np
import torch

own = False

ACTS = ("none", "relu", "relu2", "leaky_relu2", "silu", "gelu", "gelu_tanh")
BLOCK = 256                      # elements that share an 8-bit state's scale


# ------------------------------------------------------------------ cases --

def listed():
    return [
        # one token through the MLP up-projection of the 9-layer d512 model: launch latency
        dict(name="up d512, 1 token", op="epilogue", M=1, N=1536, K=512, qbits=6, act="relu2", bias="none",
             residual="none", out="bf16"),
        # the 11-layer d528 model's MLP down-projection with the residual stream, a ragged batch
        dict(name="down d528, 77 tokens", op="epilogue", M=77, N=528, K=1584, qbits=6, act="none", bias="none",
             residual="bf16", out="bf16"),
        # the int8 head of the 12-layer model (vocabulary 1792): fp32 logits for an odd number of positions
        dict(name="head 1792, 333 rows", op="epilogue", M=333, N=1792, K=512, qbits=8, act="none", bias="f32",
             residual="none", out="f32"),
        # a wide layer at a decode batch: the stream of codes
        dict(name="wide decode, 16 tokens", op="epilogue", M=16, N=16384, K=16384, qbits=6, act="silu", bias="bf16",
             residual="none", out="bf16"),
        # a long prompt through a wide layer: the tensor cores
        dict(name="wide prefill, 4096", op="epilogue", M=4096, N=8192, K=8192, qbits=6, act="gelu_tanh", bias="f32",
             residual="bf16", out="bf16"),
        # one token routed to 8 of 64 experts
        dict(name="experts, 8 of 64, 8 rows", op="grouped", M=8, E=64, active=8, pad=0, N=2048, K=2048, qbits=6,
             act="silu", bias="none", residual="none", out="bf16"),
        # a small mixture with d528 experts, three of them without a row, and a padded batch
        dict(name="experts d528, 1000 rows", op="grouped", M=1000, E=16, active=13, pad=24, N=1584, K=528, qbits=6,
             act="leaky_relu2", bias="f32", residual="none", out="bf16"),
        # a long prompt over 32 int8 experts, ragged counts
        dict(name="experts, 8192 rows", op="grouped", M=8192, E=32, active=32, pad=0, N=4096, K=2048, qbits=8,
             act="gelu", bias="bf16", residual="none", out="bf16"),
        # the vectors of one layer alone: launch latency
        dict(name="adamw, 4 vectors", op="adamw", model="vectors", n=512, tensors=4, p="f32", g="f32", bits=32,
             step=10),
        # every tensor of the 9-layer d512 model, fp32, 32-bit states
        dict(name="adamw, 9 layers, 32-bit", op="adamw", model="gpt9", n=0, tensors=0, p="f32", g="f32", bits=32,
             step=1000),
        # every matrix of the 11-layer d528 model in bf16, 8-bit states
        dict(name="adamw, 11 layers, 8-bit", op="adamw", model="unified11", n=0, tensors=0, p="bf16", g="bf16", bits=8,
             step=3),
        # one wide matrix, fp32 weights with bf16 gradients, 8-bit states: bandwidth
        dict(name="adamw, 16384x8192, 8-bit", op="adamw", model="vectors", n=16384 * 8192, tensors=1, p="f32", g="bf16",
             bits=8, step=100),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(("epilogue", "epilogue", "grouped", "grouped", "adamw"))
    if op == "adamw":
        tensors = _log(rng, 1, 40)
        return dict(op=op, model="vectors", n=_log(rng, 1, 100_000_000 // tensors), tensors=tensors,
                    p=rng.choice(("f32", "bf16")), g=rng.choice(("f32", "bf16")), bits=rng.choice((8, 32)),
                    step=_log(rng, 1, 100_000))
    out = rng.choice(("bf16", "bf16", "f32"))
    c = dict(op=op, N=_log(rng, 16, 16384), K=_log(rng, 8, 4096 if out == "f32" else 16384), qbits=rng.choice((6, 8)),
             act=rng.choice(ACTS), bias=rng.choice(("none", "f32", "bf16")),
             residual=rng.choice(("none", "none", "f32", "bf16")), out=out)
    if op == "grouped":
        c["E"] = _log(rng, 1, 128)
        while c["E"] * c["N"] * c["K"] > 1 << 28:             # the experts' codes within one wide layer's
            c["N"], c["K"] = max(16, c["N"] // 2 + 1), max(8, c["K"] // 2 + 1)
    top = max(1, min(8192, int(2.7e11 / (c["N"] * c["K"]))))  # no dearer than the listed prompt
    c["M"] = _log(rng, 1, top)
    if op == "grouped":
        c["active"] = rng.randint(1, min(c["E"], c["M"]))
        c["pad"] = rng.choice((0, 0, rng.randint(1, 64)))
    return c


# ------------------------------------------------------------- tile layout --
# Rows in tiles of 128, columns in blocks of 64; a block of a tile is
# [chunk][row][16 bytes].  int6: 16 codes u = q + 32 in three words, two codes a
# pair in the two halves of a word: pairs 0..2 at bits 0..5, pairs 3..5 at bits
# 6..11, and the low four bits of pairs 6 and 7 at bits 12..15 of words 0 and 1,
# their high two bits at bits 12..13 and 14..15 of word 2.  int8: the bytes of
# codes 0, 2, 1, 3 of each four.  Rows and columns past the end hold code 0.

def _to_tiles(q, qbits):
    E, N, K = q.shape
    rt, kb = -(-N // 128), -(-K // 64)
    full = torch.zeros((E, rt * 128, kb * 64), dtype=torch.int8, device=q.device)
    full[:, :N, :K] = q
    a = full.view(E, rt, 128, kb, 64).permute(0, 1, 3, 2, 4).contiguous()        # [E, rt, kb, row, 64]
    if qbits == 8:
        b = a.view(E, rt, kb, 128, 16, 4)[..., [0, 2, 1, 3]].reshape(E, rt, kb, 128, 4, 16)
        return b.permute(0, 1, 2, 4, 3, 5).contiguous().view(torch.uint8).view(-1)
    u = (a.to(torch.int32) + 32).view(E, rt, kb, 128, 4, 8, 2)                    # [.., group of 16, pair, half]
    p = u[..., 0] | (u[..., 1] << 16)
    lo4, hi2 = p & 0x000F000F, (p >> 4) & 0x00030003
    w = torch.stack((p[..., 0] | (p[..., 3] << 6) | (lo4[..., 6] << 12),
                     p[..., 1] | (p[..., 4] << 6) | (lo4[..., 7] << 12),
                     p[..., 2] | (p[..., 5] << 6) | (hi2[..., 6] << 12) | (hi2[..., 7] << 14)), -1)
    w = w.view(E, rt, kb, 128, 3, 4).permute(0, 1, 2, 4, 3, 5).contiguous()       # [E, rt, kb, chunk, row, word]
    return w.view(torch.uint8).view(-1)


def _from_tiles(tiles, E, N, K, qbits):
    rt, kb = -(-N // 128), -(-K // 64)
    if qbits == 8:
        b = tiles.view(torch.int8).view(E, rt, kb, 4, 128, 16).permute(0, 1, 4, 2, 3, 5).reshape(E, rt * 128, kb * 16, 4)
        return b[..., [0, 2, 1, 3]].reshape(E, rt * 128, kb * 64)[:, :N, :K]
    w = tiles.view(torch.int32).view(E, rt, kb, 3, 128, 4).permute(0, 1, 4, 2, 3, 5).reshape(E, rt * 128, kb * 4, 3)
    w0, w1, w2 = w.unbind(-1)
    six = 0x003F003F
    p = torch.stack((w0 & six, w1 & six, w2 & six, (w0 >> 6) & six, (w1 >> 6) & six, (w2 >> 6) & six,
                     ((w0 >> 12) & 0x000F000F) | ((w2 >> 8) & 0x00300030),
                     ((w1 >> 12) & 0x000F000F) | ((w2 >> 10) & 0x00300030)), -1)
    u = torch.stack((p & 63, p >> 16), -1).to(torch.int8)
    return (u - 32).reshape(E, rt * 128, kb * 64)[:, :N, :K]


# ----------------------------------------------------------------- inputs --

_DT = {"f32": torch.float32, "bf16": torch.bfloat16}


def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _offsets(case, seed):
    """Row offsets of the experts: ``active`` of them share the rows, each at least one."""
    r = np.random.default_rng(seed)
    act = np.sort(r.permutation(case["E"])[: case["active"]])
    share = r.dirichlet(np.full(case["active"], 2.0)) * (case["M"] - case["active"])
    n = np.floor(share).astype(np.int64) + 1
    n[: case["M"] - int(n.sum())] += 1
    counts = np.zeros(case["E"], np.int64)
    counts[act] = n
    return np.concatenate([[0], np.cumsum(counts)])


def _shapes(case):
    """(rows, cols) of the tensors of an AdamW case."""
    if case["model"] == "gpt9":
        layer = [(512, 512), (256, 512), (256, 512), (512, 512), (1536, 512), (512, 1536), (1, 512), (1, 512)]
        return [(1024, 512)] + layer * 9
    if case["model"] == "unified11":
        return [(1584, 528), (528, 528), (1584, 528), (528, 1584)] * 11
    return [(1, case["n"])] * case["tensors"]


def prepare(case, seed):
    g = _gen(seed)
    rand = lambda *s: torch.randn(*s, device="cuda", generator=g)  # noqa: E731
    if case["op"] == "adamw":
        # views of one buffer a kind, as an optimizer lays its state out; each starts on a block of 256
        shapes = _shapes(case)
        sizes = [a * b for a, b in shapes]
        at = np.concatenate([[0], np.cumsum([-(-n // BLOCK) * BLOCK for n in sizes])]).tolist()
        total = at[-1]
        p = (rand(total) * 0.02).to(_DT[case["p"]])
        grad = (rand(total) * torch.exp(rand(total))).mul_(1e-3).to(_DT[case["g"]])
        if case["bits"] == 32:
            m, v = rand(total).mul_(1e-3), (rand(total) * 1e-3).square_().add_(1e-8)
            ms = vs = None
        else:
            m = torch.randint(-127, 128, (total,), device="cuda", generator=g, dtype=torch.int8)
            v = torch.randint(1, 256, (total,), device="cuda", generator=g, dtype=torch.uint8)
            ms = torch.rand(total // BLOCK, device="cuda", generator=g).add_(0.5).mul_(3e-3 / 127)
            vs = torch.rand(total // BLOCK, device="cuda", generator=g).add_(0.5).mul_(9e-6 / 255 ** 4)
        real = torch.cat([torch.arange(a, a + n, device="cuda") for a, n in zip(at, sizes)])
        for t in (p, grad, m, v):                              # nothing between the tensors
            kept = t[real]
            t.zero_()[real] = kept
        cut = lambda t, q: [t[a // q:a // q + -(-n // q)] for a, n in zip(at, sizes)]  # noqa: E731
        s = dict(case=case, p=p, g=grad, m=m, v=v, ms=ms, vs=vs, step=case["step"], seed=seed & 0x7FFFFFFF,
                 sizes=torch.tensor(at, device="cuda").diff(),
                 wd=[0.0 if a == 1 and case["model"] == "gpt9" else 0.1 for a, _ in shapes])
        s["lists"] = dict(params=cut(p, 1), grads=cut(grad, 1), exp_avgs=cut(m, 1), exp_avg_sqs=cut(v, 1),
                          scales=None if ms is None else (cut(ms, BLOCK), cut(vs, BLOCK)))
        return s
    E, M, N, K = case.get("E", 1), case["M"], case["N"], case["K"]
    rows = M + case.get("pad", 0)
    top = 31 if case["qbits"] == 6 else 127
    q = (rand(E, N, K) * (top / 4)).round_().clamp_(-top, top).to(torch.int8)
    s = dict(case=case, tiles=_to_tiles(q, case["qbits"]).view(E, -1),
             scale=((torch.rand(E, N, device="cuda", generator=g) + 0.5) * (4.0 / top / math.sqrt(K))).half())
    del q
    x = rand(rows, -(-K // 8) * 8)                             # rows start on 16 bytes, as activations do
    s["x"] = x.to(torch.bfloat16)[:, :K]
    s["bias"] = None if case["bias"] == "none" else (rand(E, N) * 0.1).to(_DT[case["bias"]])
    s["residual"] = None if case["residual"] == "none" else rand(rows, N).to(_DT[case["residual"]])
    if case["op"] == "grouped":
        off = _offsets(case, seed)
        s["offsets"], s["off"] = torch.from_numpy(off.astype(np.int32)).cuda(), off.tolist()
        s["y"] = torch.zeros((rows, N), dtype=_DT[case["out"]], device="cuda")   # rows past the last expert's stay 0
    else:
        s["tiles"], s["scale"] = s["tiles"][0], s["scale"][0]
        s["bias"] = None if s["bias"] is None else s["bias"][0]
    return s


# ------------------------------------------------------------ plain forms --

def _act(z, act):
    if act == "relu":
        return torch.where(z > 0, z, torch.zeros_like(z))
    if act == "relu2":
        z = torch.where(z > 0, z, torch.zeros_like(z))
        return z * z
    if act == "leaky_relu2":
        z = torch.where(z > 0, z, 0.5 * z)
        return z * z
    if act == "silu":
        return z / (1 + torch.exp(-z))
    if act == "gelu":
        return 0.5 * z * (1 + torch.erf(z * math.sqrt(0.5)))
    if act == "gelu_tanh":
        return 0.5 * z * (1 + torch.tanh(math.sqrt(2 / math.pi) * (z + 0.044715 * z * z * z)))
    return z


def _layer(x, w, scale, bias, residual, act, out):
    z = (x.float() @ w.t()) * scale.float()
    if bias is not None:
        z = z + bias.float()
    y = _act(z, act)
    if residual is not None:
        y = y + residual.float()
    return y.to(out)


def _plain_epilogue(s):
    c = s["case"]
    w = _from_tiles(s["tiles"], 1, c["N"], c["K"], c["qbits"])[0].float()
    return _layer(s["x"], w, s["scale"], s["bias"], s["residual"], c["act"], _DT[c["out"]])


def _plain_grouped(s):
    c, off, y = s["case"], s["off"], s["y"]
    for e in range(c["E"]):
        a, b = off[e], off[e + 1]
        if a < b:
            w = _from_tiles(s["tiles"][e], 1, c["N"], c["K"], c["qbits"])[0].float()
            y[a:b] = _layer(s["x"][a:b], w, s["scale"][e], None if s["bias"] is None else s["bias"][e],
                            None if s["residual"] is None else s["residual"][a:b], c["act"], y.dtype)
    return y


BETA1, BETA2, EPS, LR = 0.9, 0.95, 1e-8, 1e-3


def _f(x):
    return float(np.float32(x))


def _hash(index, key):
    """32 random bits for each element, in 64-bit integers: two multiply-xorshift rounds over its index and the key."""
    mask = 0xFFFFFFFF
    z = ((index & mask) * 0x9E3779B9 + (index >> 32) * 0x7FEB3529 + key) & mask
    z = ((z ^ (z >> 16)) * 0x21F0AAAD) & mask
    z = ((z ^ (z >> 15)) * 0x735A2D97) & mask
    return z ^ (z >> 15)


def _fourth(q):
    t = q * q
    return t * t


def _plain_adamw(s):
    """All tensors as the one buffer that holds them (what lies between two tensors is zero and stays so), in place;
    every line is one rounding to 32 bits."""
    step, sizes = s["step"], s["sizes"]
    p, m, v, ms, vs = s["p"], s["m"], s["v"], s["ms"], s["vs"]
    g = s["g"].float()
    decay = torch.tensor([_f(1 - LR * w) for w in s["wd"]], device="cuda").repeat_interleave(sizes)
    m32 = m.float() if ms is None else (m.view(-1, BLOCK).float() * ms[:, None]).view(-1)
    v32 = v.float() if vs is None else (_fourth(v.view(-1, BLOCK).float()) * vs[:, None]).view(-1)
    m32 = m32 * _f(BETA1) + g * _f(1 - BETA1)
    v32 = v32 * _f(BETA2) + (g * g) * _f(1 - BETA2)
    d = torch.sqrt(v32) * _f(1 / math.sqrt(1 - BETA2 ** step)) + _f(EPS)
    u = (m32 / d) * _f(LR / (1 - BETA1 ** step))
    p.copy_(p.float() * decay - u)
    if ms is None:
        m.copy_(m32)
        v.copy_(v32)
        return
    tensor = torch.arange(len(s["wd"]), device="cuda")
    key = (s["seed"] + step * 0x632BE5AB + tensor * 0x2C1B3C6D) & 0xFFFFFFFF
    index = torch.arange(p.numel(), device="cuda") - (sizes.cumsum(0) - sizes).repeat_interleave(sizes)
    z = _hash(index, key.repeat_interleave(sizes)).view(-1, BLOCK)
    um, uv = (z >> 16).float() * 2.0 ** -16, (z & 0xFFFF).float() * 2.0 ** -16
    mb, vb = m32.view(-1, BLOCK), v32.view(-1, BLOCK)
    am, av = mb.abs().amax(1), vb.amax(1)
    keep_m, keep_v = am >= 2.0 ** -80, av >= 2.0 ** -80
    zero = torch.zeros_like(am)
    im = torch.where(keep_m, torch.full_like(am, 127.0) / am, zero)[:, None]
    iv = torch.where(keep_v, torch.full_like(av, 255.0 ** 4) / av, zero)[:, None]
    qm = torch.floor(mb * im + um).clamp(-127, 127)
    x = vb * iv
    q0 = torch.floor(torch.sqrt(torch.sqrt(x)))               # then set right against the fourth powers themselves
    q0 = torch.where(_fourth(q0) > x, q0 - 1, q0)
    q0 = torch.where(_fourth(q0 + 1) <= x, q0 + 1, q0).clamp(0, 254)
    lo, hi = _fourth(q0), _fourth(q0 + 1)
    qv = torch.where(uv * (hi - lo) < x - lo, q0 + 1, q0)
    qv = torch.where((x > 0) & (qv == 0), torch.ones_like(qv), qv)
    m.copy_(qm.view(-1))
    v.copy_(qv.view(-1))
    ms.copy_(torch.where(keep_m, am * _f(1 / 127), zero))
    vs.copy_(torch.where(keep_v, av * _f(1 / 255.0 ** 4), zero))


# -------------------------------------------------------------------- run --

def run(state):
    c = state["case"]
    if own:
        from int6_int8_weight_b200 import gq
        if c["op"] == "epilogue":
            return gq.gemm_epilogue(state["x"], state["tiles"], state["scale"], c["qbits"], bias=state["bias"],
                                    act=c["act"], residual=state["residual"], out_dtype=_DT[c["out"]])
        if c["op"] == "grouped":
            return gq.gemm_grouped(state["x"], state["offsets"], state["tiles"], state["scale"], c["qbits"],
                                   bias=state["bias"], act=c["act"], residual=state["residual"], y=state["y"])
        gq.adamw_step(**state["lists"], step=state["step"], lr=LR, betas=(BETA1, BETA2), eps=EPS,
                      weight_decay=state["wd"], seed=state["seed"])
    elif c["op"] == "epilogue":
        return _plain_epilogue(state)
    elif c["op"] == "grouped":
        return _plain_grouped(state)
    else:
        _plain_adamw(state)
    # the state itself: 32-bit values, or codes (whole numbers) and their blocks' scales
    return {k: state[k] for k in ("p", "m", "v", "ms", "vs") if state[k] is not None}


def work(case):
    if case["op"] == "adamw":
        n = sum(a * b for a, b in _shapes(case))
        pb, gb = (4 if case[k] == "f32" else 2 for k in ("p", "g"))
        per = 2 * pb + gb + (16 if case["bits"] == 32 else 4 + 16 / BLOCK)
        return {"bytes": n * per, "flops": 16 * n}
    M, N, K = case["M"], case["N"], case["K"]
    size = {"none": 0, "f32": 4, "bf16": 2}
    held = case.get("active", 1) * N * (K * (0.75 if case["qbits"] == 6 else 1) + 2 + size[case["bias"]])
    return {"bytes": held + M * K * 2 + M * N * (size[case["residual"]] + size[case["out"]]), "flops": 2 * M * N * K}


def exact(case, seed):
    """In 64 bits, from the definitions.  An 8-bit state's codes are rounded by random numbers: only the weights have a value."""
    s = prepare(case, seed)
    if case["op"] == "epilogue":
        return _exact_layer(case, s["x"], s["tiles"], s["scale"], s["bias"], s["residual"])
    if case["op"] == "grouped":
        off = s["off"]
        y = torch.zeros(s["y"].shape, dtype=torch.float64, device="cuda")
        for e in range(case["E"]):
            a, b = off[e], off[e + 1]
            if a < b:
                y[a:b] = _exact_layer(case, s["x"][a:b], s["tiles"][e], s["scale"][e],
                                      None if s["bias"] is None else s["bias"][e],
                                      None if s["residual"] is None else s["residual"][a:b])
        return y
    p = s["p"].double()
    t, step = s["lists"], case["step"]
    m64, v64 = s["m"].double(), s["v"].double()
    if case["bits"] == 8:
        m64 = m64 * s["ms"].double().repeat_interleave(BLOCK)
        v64 = v64 ** 4 * s["vs"].double().repeat_interleave(BLOCK)
    at = 0
    for q, g, wd in zip(t["params"], t["grads"], s["wd"]):
        k = slice(at, at + q.numel())
        g = g.double()
        m64[k] = BETA1 * m64[k] + (1 - BETA1) * g
        v64[k] = BETA2 * v64[k] + (1 - BETA2) * g ** 2
        mean, var = m64[k] / (1 - BETA1 ** step), v64[k] / (1 - BETA2 ** step)
        p[k] = p[k] * (1 - LR * wd) - LR * mean / (var.sqrt() + EPS)
        at += -(-q.numel() // BLOCK) * BLOCK
    if case["bits"] == 8:
        return {"p": p, "m": None, "v": None, "ms": None, "vs": None}
    return {"p": p, "m": m64, "v": v64}


def _exact_layer(case, x, tiles, scale, bias, residual):
    N, K = case["N"], case["K"]
    t = tiles.long().view(-1, -(-K // 64), 3 if case["qbits"] == 6 else 4, 128, 16)   # [row tile, block, chunk, row, byte]
    t = t.permute(0, 3, 1, 2, 4).reshape(t.shape[0] * 128, -(-K // 64), -1)[:N]       # each row's bytes of each block
    if case["qbits"] == 8:
        k = torch.arange(64, device="cuda")
        q = t[..., k // 4 * 4 + torch.tensor([0, 2, 1, 3], device="cuda")[k % 4]]
        q = torch.where(q > 127, q - 256, q)
    else:
        # bit b of code k of a block, found one at a time
        q = torch.full((N, t.shape[1], 64), -32, dtype=torch.int64, device="cuda")
        k = torch.arange(64, device="cuda")
        pair, half = k % 16 // 2, k % 2
        for bit in range(6):
            word = torch.where(pair < 6, pair % 3, torch.full_like(pair, 2) if bit > 3 else pair - 6)
            low = torch.where(pair < 3, bit, 6 + bit)
            low = torch.where(pair >= 6, 12 + bit if bit < 4 else 12 + 2 * (pair - 6) + bit - 4, low)
            place = (k // 16 * 3 + word) * 32 + half * 16 + low
            q += ((t[..., place // 8] >> (place % 8)) & 1) << bit
    w = q.reshape(N, -1)[:, :K].double() * scale.double()[:, None]
    z = x.double() @ w.t()
    if bias is not None:
        z += bias.double()
    act = case["act"]
    if act in ("relu", "relu2"):
        z = z.clamp(min=0) ** (1 if act == "relu" else 2)
    elif act == "leaky_relu2":
        z = torch.maximum(z, z / 2) ** 2
    elif act == "silu":
        z = z * torch.sigmoid(z)
    elif act == "gelu":
        z = z * torch.special.ndtr(z)
    elif act == "gelu_tanh":
        z = z * torch.sigmoid(2 * math.sqrt(2 / math.pi) * (z + 0.044715 * z ** 3))
    return z if residual is None else z + residual.double()
