"""What a training step of the adapters needs around the layers, measured: the norm in front of them, the loss
through the output head, the optimizer.

Formulas:
  norm_fwd   h = bf16(x + res);  rstd = 1 / sqrt(mean(h^2) + eps);  y = bf16(h rstd w);  8 bits: per row and 128
             columns of y, e the least integer (>= -127) with max |y| 2^-e <= 448, codes = e4m3(y 2^-e), byte e + 127
  norm_bwd   dh = bf16(dres + rstd (w dy - h rstd^2 mean(w dy h)));  dw = sum over rows of dy h rstd
  head       l = X W^T;  lse = log sum exp l;  loss = lse - l_label (0 without a label);
             dX = dloss (softmax(l) W - W_label) (0 without a label)
  adamw      g = s grad;  m' = b1 m + (1 - b1) g;  v' = b2 v + (1 - b2) g^2;
             p' = p - lr wd p - lr / (1 - b1^t) m' / (sqrt(v') / sqrt(1 - b2^t) + eps)
             8 bits: m and sqrt(v) as e4m3 with a power-of-two scale per 128 values, rounded down after the
             addition of a noise below one step, noise = (byte + 1/2) / 256; a v that is not 0 stays so
"""

import math

import numpy as np
import torch

own = False

BLOCK = 128           # values (a row's columns, a tensor's elements) that share one 8-bit scale
E4M3_MAX = 448.0
NF4_BLOCK = 64        # weights per absmax
NF4_GROUP = 256       # absmax values per double-quantization scale
NF4_LEVELS = [-1.0, -0.6961928009986877, -0.5250730514526367, -0.39491748809814453, -0.28444138169288635,
              -0.18477343022823334, -0.09105002880096436, 0.0, 0.07958029955625534, 0.16093020141124725,
              0.24611230194568634, 0.33791524171829224, 0.44070982933044434, 0.5626169443130493,
              0.7229568362236023, 1.0]
BETA1, BETA2, ADAM_EPS, DECAY, RATE = 0.9, 0.999, 1e-8, 0.01, 2e-4
NORM_EPS = 1e-6


def listed():
    return [
        # one token of a decode step in front of an 8-bit layer: latency
        {"name": "norm_fwd_1x4096", "op": "norm_fwd", "T": 1, "H": 4096, "res": True, "rows8": True, "y16": True},
        # a training batch in front of an 8-bit layer with an adapter
        {"name": "norm_fwd_8192x8192", "op": "norm_fwd", "T": 8192, "H": 8192, "res": True, "rows8": True, "y16": True},
        # a short sequence back through a trained norm, nothing a multiple of a tile
        {"name": "norm_bwd_301x4160", "op": "norm_bwd", "T": 301, "H": 4160, "dres": True, "dw": True},
        # a training batch back through a trained norm
        {"name": "norm_bwd_8192x4096", "op": "norm_bwd", "T": 8192, "H": 4096, "dres": True, "dw": True},
        # one token scored against a small vocabulary
        {"name": "loss_1x32000x4096", "op": "head", "T": 1, "V": 32000, "H": 4096, "W": "bf16", "grad": False},
        # a held-out batch scored through a 4-bit head
        {"name": "loss_1024x65536x4096_nf4", "op": "head", "T": 1024, "V": 65536, "H": 4096, "W": "nf4", "grad": False},
        # a short sequence, a vocabulary that is no multiple of anything
        {"name": "grad_301x50021x2304", "op": "head", "T": 301, "V": 50021, "H": 2304, "W": "bf16", "grad": True},
        # a training batch through an 8-bit head
        {"name": "grad_2048x65536x4096_fp8", "op": "head", "T": 2048, "V": 65536, "H": 4096, "W": "fp8", "grad": True},
        # a training batch through a 16-bit head with a large vocabulary
        {"name": "grad_4096x128000x4096", "op": "head", "T": 4096, "V": 128000, "H": 4096, "W": "bf16", "grad": True},
        # one projection's two adapter factors: launch latency
        {"name": "adamw32_1_layer_pair", "op": "adamw", "bits": 32, "layers": 1, "kinds": 1, "hidden": 4096,
         "inter": 14336, "r": 16, "scaled": False},
        # the factors of all seven projections of 32 layers, states in 32 bits
        {"name": "adamw32_448_tensors", "op": "adamw", "bits": 32, "layers": 32, "kinds": 7, "hidden": 4096,
         "inter": 14336, "r": 16, "scaled": True},
        # the same with states in 8 bits
        {"name": "adamw8_448_tensors", "op": "adamw", "bits": 8, "layers": 32, "kinds": 7, "hidden": 4096,
         "inter": 14336, "r": 16, "scaled": True},
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _log_64(rng, lo, hi):
    return 64 * max(1, _log_int(rng, lo, hi) // 64)


def draw(rng):
    op = rng.choice(["norm_fwd", "norm_bwd", "head", "head", "head", "adamw", "adamw"])
    if op in ("norm_fwd", "norm_bwd"):
        H = _log_64(rng, 64, 16384)
        T = min(_log_int(rng, 1, 16384), (1 << 26) // H)
        if op == "norm_bwd":
            return {"op": op, "T": T, "H": H, "dres": rng.random() < 0.7, "dw": rng.random() < 0.7}
        rows8 = rng.random() < 0.7
        return {"op": op, "T": T, "H": H, "res": rng.random() < 0.7, "rows8": rows8,
                "y16": not rows8 or rng.random() < 0.7}
    if op == "head":
        W = rng.choice(["bf16", "bf16", "nf4", "fp8"])
        H, V = _log_64(rng, 256, 8192), _log_int(rng, 500, 160000)
        V = min(V, 560_000_000 // H)
        V = V if W == "bf16" else 64 * (V // 64)
        T = min(_log_int(rng, 1, 4096), 4096 * 128000 * 4096 // (V * H))
        return {"op": op, "T": T, "V": V, "H": H, "W": W, "grad": rng.random() < 0.7}
    return {"op": op, "bits": rng.choice([32, 8]), "layers": rng.randint(1, 32), "kinds": rng.randint(1, 7),
            "hidden": _log_int(rng, 65, 4096), "inter": _log_int(rng, 100, 14336), "r": rng.choice([1, 4, 8, 15, 16]),
            "scaled": rng.random() < 0.5}


# ------------------------------------------------------------------ inputs
def _normal(gen, shape, std=1.0):
    return torch.randn(shape, generator=gen, device="cuda", dtype=torch.float32) * std


def _uniform(gen, shape):
    return torch.rand(shape, generator=gen, device="cuda", dtype=torch.float32)


def _bf16(gen, shape, std=1.0):
    return _normal(gen, shape, std).to(torch.bfloat16)


def _nf4_weight(w):
    """Codes, 8-bit absmax and group scales of a weight [rows, cols]."""
    n, (rows, cols) = w.numel(), w.shape
    b = w.reshape(n // NF4_BLOCK, NF4_BLOCK)
    absmax = b.abs().amax(1)
    levels = torch.tensor(NF4_LEVELS, device="cuda")
    c = torch.bucketize(b / absmax[:, None], (levels[1:] + levels[:-1]) / 2, out_int32=True)
    c = c.to(torch.uint8).view(-1, 2)
    groups = -(-absmax.numel() // NF4_GROUP)
    pad = torch.zeros(groups * NF4_GROUP, device="cuda")
    pad[:absmax.numel()] = absmax
    scale = pad.view(groups, NF4_GROUP).amax(1)
    q = torch.round(pad.view(groups, NF4_GROUP) / scale[:, None] * 255).to(torch.uint8).view(-1)[:absmax.numel()]
    return {"codes": c[:, 0] | (c[:, 1] << 4), "q": q.contiguous(), "scale": scale, "rows": rows, "cols": cols}


def _fp8_weight(w):
    """Codes and scale bytes of a weight, one per 128 x 128 block."""
    R, C = w.shape
    p = torch.zeros((-(-R // BLOCK) * BLOCK, -(-C // BLOCK) * BLOCK), device="cuda")
    p[:R, :C] = w
    b = p.view(p.shape[0] // BLOCK, BLOCK, p.shape[1] // BLOCK, BLOCK)
    e = _exponent(b.abs().amax((1, 3)))
    c = (b * _pow2(-e)[:, None, :, None]).to(torch.float8_e4m3fn).view(torch.uint8)
    return {"codes": c.view(p.shape)[:R, :C].contiguous(), "scales": (e + 127).to(torch.uint8), "rows": R, "cols": C}


def _adapter_shapes(case):
    """Both factors of the adapters of a model's projections: q, k, v, o, gate, up, down of each layer."""
    h, i, r = case["hidden"], case["inter"], case["r"]
    kv = max(1, h // 4)
    sides = [(h, h), (h, kv), (h, kv), (h, h), (h, i), (h, i), (i, h)][:case["kinds"]]
    return [s for a, b in sides for s in ((r, a), (b, r))] * case["layers"]


def _adapters(case, gen, st):
    """All tensors in one buffer of each kind, every tensor starting at a multiple of 128 values."""
    shapes = _adapter_shapes(case)
    pitch = [-(-a * b // BLOCK) * BLOCK for a, b in shapes]
    off = np.cumsum([0] + pitch[:-1]).tolist()
    N = sum(pitch)
    live = torch.zeros(N, device="cuda")
    size = torch.empty(N, device="cuda")
    for k, (a, b) in enumerate(shapes):
        live[off[k]:off[k] + a * b] = 1.0
        size[off[k]:off[k] + pitch[k]] = 10.0 ** (-2.0 - (k * 7 % 5) * 0.5)  # some adapters' gradients are far smaller
    st["shapes"], st["off"], st["N"] = shapes, off, N
    st["master"] = _normal(gen, N, 0.01) * live
    st["param"] = st["master"].to(torch.bfloat16)
    spread = torch.exp(_normal(gen, N, 1.0))  # an element's gradients have a size of their own
    st["grad"] = _normal(gen, N) * size * spread * live
    m = _normal(gen, N, 0.25) * size * spread * live
    v = (size * spread * (0.6 + 0.8 * _uniform(gen, N))).square() * live
    if case["bits"] == 32:
        st["m"], st["v"] = m, v
    else:
        for name, x in (("m", m), ("v", v.sqrt())):
            b = x.view(-1, BLOCK)
            e = _exponent(b.abs().amax(1))
            st[name] = (b * _pow2(-e)[:, None]).to(torch.float8_e4m3fn).view(torch.uint8).view(-1)
            st[name + "_scales"] = (e + 127).to(torch.uint8)
    st["t"] = 100
    st["seed"] = int(torch.randint(0, 1 << 31, (1,), generator=gen, device="cuda"))
    st["scale"] = 0.25 + 0.75 * _uniform(gen, 1) if case["scaled"] else None  # what clips the gradients' norm


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    op = case["op"]
    st = dict(case)
    if op == "adamw":
        _adapters(case, gen, st)
        return st
    T, H = case["T"], case["H"]
    if op in ("norm_fwd", "norm_bwd"):
        # rows of several sizes, as a residual stream has them, and a few columns far above the others
        col = torch.exp(_normal(gen, H, 0.5)) * (1 + 30 * (_uniform(gen, H) < 0.003))
        row = torch.exp(_normal(gen, (T, 1), 0.7))
        h = (_normal(gen, (T, H)) * row * col).to(torch.bfloat16)
        st["w"] = 1 + _normal(gen, H, 0.2)
        if op == "norm_fwd":
            st["x"] = h
            st["r"] = _bf16(gen, (T, H)) if case["res"] else None
        else:
            st["h"] = h
            st["rstd"] = torch.rsqrt(h.float().square().mean(1) + NORM_EPS)
            st["dy"] = _bf16(gen, (T, H))
            st["dr"] = _bf16(gen, (T, H)) if case["dres"] else None
        return st
    V = case["V"]
    w = torch.empty((V, H), device="cuda")
    for a in range(0, V, 1 << 15):
        b = min(V, a + (1 << 15))
        w[a:b] = _normal(gen, (b - a, H), 0.02)
    labels = torch.randint(0, V, (T,), generator=gen, device="cuda")
    # from rows that know nothing of their label to rows that are nearly sure of it
    sure = 15.0 * _uniform(gen, (T, 1)) / (H * 0.02 ** 2)
    st["X"] = (_normal(gen, (T, H)) * min(1.0, 64 / math.sqrt(H)) + sure * w[labels]).to(torch.bfloat16)
    st["W16"] = w.to(torch.bfloat16) if case["W"] == "bf16" else None
    st["W4"] = _nf4_weight(w) if case["W"] == "nf4" else None
    st["W8"] = _fp8_weight(w) if case["W"] == "fp8" else None
    st["labels"] = torch.where(_uniform(gen, T) < 0.1, torch.full_like(labels, -100), labels)  # prompts carry none
    st["dloss"] = (_uniform(gen, T) + 0.5) / T
    return st


# ------------------------------------------------------------------ plain forms
def _exponent(a):
    """The least e with a 2^-e <= 448, at least -127; -127 for a = 0."""
    m, p = torch.frexp(a)  # a = m 2^p, 0.5 <= m < 1; 448 = 0.875 * 2^9
    e = torch.where(m <= 0.875, p - 9, p - 8)
    return torch.where(a == 0, torch.full_like(e, -127), e.clamp_min(-127))


def _pow2(e):
    """2^e in fp32, exact, for whole e from -127 to 127 (-127: the subnormal one)."""
    e = e.to(torch.int32)
    return torch.where(e < -126, torch.full_like(e, 1 << 22), (e + 127) << 23).view(torch.float32)


def _rows8(y):
    """Codes of rows [T, H], padded with 0 to whole blocks, and scale bytes by groups of four blocks: [ceil(H / 512), T, 4]."""
    T, H = y.shape
    blocks, groups = -(-H // BLOCK), -(-H // (4 * BLOCK))
    p = torch.zeros((T, blocks * BLOCK), device=y.device)
    p[:, :H] = y.float()
    b = p.view(T, blocks, BLOCK)
    e = _exponent(b.abs().amax(2))
    codes = (b * _pow2(-e)[:, :, None]).to(torch.float8_e4m3fn).view(T, blocks * BLOCK)
    s = torch.zeros((T, groups * 4), dtype=torch.uint8, device=y.device)
    s[:, :blocks] = (e + 127).to(torch.uint8)
    return codes, s.view(T, groups, 4).permute(1, 0, 2).contiguous().view(torch.float8_e8m0fnu)


def _norm_fwd(st):
    h = st["x"].float()
    if st["r"] is not None:
        h = h + st["r"].float()
    h16 = h.to(torch.bfloat16)
    h = h16.float()
    rstd = torch.rsqrt(h.square().mean(1) + NORM_EPS)
    y = (h * rstd[:, None] * st["w"]).to(torch.bfloat16)
    out = {"rstd": rstd}
    if st["r"] is not None:
        out["h"] = h16
    if st["y16"]:
        out["y"] = y
    if st["rows8"]:
        out["codes"], out["scales"] = _rows8(y)
    return out


def _norm_bwd(st):
    h, dy, rstd = st["h"].float(), st["dy"].float(), st["rstd"][:, None]
    g = dy * st["w"]
    n = h * rstd
    dh = rstd * (g - n * (g * n).mean(1, keepdim=True))
    if st["dr"] is not None:
        dh = dh + st["dr"].float()
    out = {"dh": dh.to(torch.bfloat16)}
    if st["dw"]:
        out["dw"] = (dy * n).sum(0)
    return out


def _head_weight(st):
    """The head's values in fp32: bf16 as they are, or bf16(level * absmax), or code 2^e."""
    if st["W16"] is not None:
        return st["W16"].float()
    if st["W8"] is not None:
        w = st["W8"]
        R, C = w["rows"], w["cols"]
        p = torch.zeros((-(-R // BLOCK) * BLOCK, -(-C // BLOCK) * BLOCK), device="cuda")
        p[:R, :C] = w["codes"].view(torch.float8_e4m3fn).float()
        b = p.view(p.shape[0] // BLOCK, BLOCK, p.shape[1] // BLOCK, BLOCK)
        b *= _pow2(w["scales"].to(torch.int32) - 127)[:, None, :, None]
        return p[:R, :C]
    w = st["W4"]
    c = torch.stack((w["codes"] & 15, w["codes"] >> 4), 1).view(-1)
    v = torch.index_select(torch.tensor(NF4_LEVELS, device="cuda"), 0, c.int()).view(-1, NF4_BLOCK)
    ratio = w["q"].float() / 255.0
    a = ratio * w["scale"].repeat_interleave(NF4_GROUP)[:ratio.numel()]
    return (v * a[:, None]).to(torch.bfloat16).float().view(w["rows"], w["cols"])


def _head(st):
    W, X, y = _head_weight(st), st["X"].float(), st["labels"]
    has = (y >= 0) & (y < st["V"])
    at = torch.where(has, y, torch.zeros_like(y))[:, None]
    l = X @ W.t()
    top = l.amax(1, keepdim=True)
    target = l.gather(1, at)
    p = torch.exp(l - top)
    del l
    # the sum over the others, so that a small loss and 1 - p keep their digits
    mine = p.gather(1, at)
    p.scatter_(1, at, 0.0)
    others = p.sum(1, keepdim=True)
    total = others + mine
    loss = torch.where(mine > 0, torch.log1p(others / mine), top + torch.log(total) - target)[:, 0]
    out = {"loss": torch.where(has, loss, torch.zeros_like(loss)), "lse": (top + torch.log(total))[:, 0]}
    if st["grad"]:
        p = p / total
        p.scatter_(1, at, -others / total)
        out["dX"] = ((p @ W) * torch.where(has, st["dloss"], torch.zeros_like(loss))[:, None]).to(torch.bfloat16)
    return out


def _noise(N, seed, device):
    """Two numbers in (0, 1) for each of N values: (byte + 1/2) / 256 of a hash of the pair's number and the seed."""
    def mix(x):
        x = x ^ (x >> 16)
        x = (x * 0x85ebca6b) & 0xffffffff
        x = x ^ (x >> 13)
        x = (x * 0xc2b2ae35) & 0xffffffff
        return x ^ (x >> 16)
    key = mix(torch.tensor(seed, dtype=torch.int64, device=device))
    x = mix(torch.arange(N // 2, dtype=torch.int64, device=device) ^ key)
    u = torch.stack((x & 255, (x >> 8) & 255, (x >> 16) & 255, x >> 24), 1).view(N, 2)
    return (u.float() + 0.5) / 256


def _to8(x, u, keep):
    """Codes and scale bytes of x by blocks, rounded down after the addition of u steps; keep: what is not 0 stays so."""
    b = x.view(-1, BLOCK)
    e = _exponent(b.abs().amax(1))
    y = (b * _pow2(-e)[:, None]).double()
    _, p = torch.frexp(y)
    step = torch.exp2((p - 1).clamp_min(-6).double() - 3)
    n = torch.floor(y.abs() / step + u.view(-1, BLOCK))
    if keep:
        n = torch.where(y != 0, n.clamp_min(1), n)
    c = torch.copysign(n * step, y).float().to(torch.float8_e4m3fn)
    return c.view(torch.uint8).view(-1), (e + 127).to(torch.uint8)


def _from8(codes, scales):
    return (codes.view(torch.float8_e4m3fn).float().view(-1, BLOCK) * _pow2(scales.to(torch.int32) - 127)[:, None]).view(-1)


def _adamw(st):
    g = st["grad"]
    if st["scale"] is not None:
        g = g * st["scale"]
    small = st["bits"] == 8
    m, v = (_from8(st["m"], st["m_scales"]), _from8(st["v"], st["v_scales"]).square()) if small else (st["m"], st["v"])
    m = BETA1 * m + (1 - BETA1) * g
    v = BETA2 * v + (1 - BETA2) * (g * g)
    root = torch.sqrt(v)
    p = st["master"]
    rate = RATE / (1 - BETA1 ** st["t"])
    p = p - RATE * DECAY * p - rate * (m / (root * (1 / math.sqrt(1 - BETA2 ** st["t"])) + ADAM_EPS))
    st["master"].copy_(p)
    st["param"].copy_(p)
    if small:
        u = _noise(st["N"], st["seed"], g.device)
        for name, x, k in (("m", m, 0), ("v", root, 1)):
            c, s = _to8(x, u[:, k], k == 1)
            st[name].copy_(c)
            st[name + "_scales"].copy_(s)
    else:
        st["m"].copy_(m)
        st["v"].copy_(v)
    return _adamw_out(st)


def _adamw_out(st):
    out = {"param": st["param"], "master": st["master"]}
    if st["bits"] == 32:
        return {**out, "m": st["m"], "v": st["v"]}
    for name in ("m", "v"):
        out[name] = st[name].view(torch.float8_e4m3fn)
        out[name + "_scales"] = st[name + "_scales"].view(torch.float8_e8m0fnu)
    return out


def _run_plain(st):
    return {"norm_fwd": _norm_fwd, "norm_bwd": _norm_bwd, "head": _head, "adamw": _adamw}[st["op"]](st)


# ------------------------------------------------------------------ the framework's operators
def _run_own(st):
    import bit_nf4_quantized_20_amd as q
    op = st["op"]
    if op == "norm_fwd":
        y, rows, h, rstd = q.qlora_rmsnorm_fwd(st["x"], st["w"], residual=st["r"], eps=NORM_EPS, y16=st["y16"],
                                               rows8=st["rows8"])
        out = {"rstd": rstd}
        if st["r"] is not None:
            out["h"] = h
        if st["y16"]:
            out["y"] = y
        if st["rows8"]:
            out["codes"] = rows.codes.view(torch.float8_e4m3fn)
            out["scales"] = rows.scales[:, :st["T"]].view(torch.float8_e8m0fnu)
        return out
    if op == "norm_bwd":
        dh, dw = q.qlora_rmsnorm_bwd(st["dy"], st["h"], st["w"], st["rstd"], dres=st["dr"], want_dweight=st["dw"])
        return {"dh": dh, "dw": dw} if st["dw"] else {"dh": dh}
    if op == "head":
        W, w4, w8 = st["W16"], st["W4"], st["W8"]
        if w4 is not None:
            W = q.NF4Weight(w4["codes"], w4["q"], w4["scale"], w4["rows"], w4["cols"])
        if w8 is not None:
            W = q.FP8Weight(w8["codes"], w8["scales"], w8["rows"], w8["cols"])
        if not st["grad"]:
            loss, lse = q.qlora_head_loss(W, st["X"], st["labels"])
            return {"loss": loss, "lse": lse}
        loss, lse, dX = q.qlora_head_loss_grad(W, st["X"], st["labels"], st["dloss"])
        return {"loss": loss, "lse": lse, "dX": dX}
    if "plan" not in st:  # a program makes it once, with its adapters
        def parts(t):
            return [t[o:o + a * b].view(a, b) for o, (a, b) in zip(st["off"], st["shapes"])]
        states = q.AdamWState(st["m"], st["v"], st.get("m_scales"), st.get("v_scales"))
        st["plan"] = q.qlora_adamw_plan(parts(st["param"]), parts(st["master"]), parts(st["grad"]), states)
    q.qlora_adamw_step(st["plan"], st["t"], lr=RATE, beta1=BETA1, beta2=BETA2, eps=ADAM_EPS, weight_decay=DECAY,
                       grad_scale=st["scale"], seed=st["seed"])
    return _adamw_out(st)


def run(state):
    return _run_own(state) if own else _run_plain(state)


# ------------------------------------------------------------------ what a pass cannot do without
def work(case):
    op = case["op"]
    if op == "adamw":  # parameters, their 16-bit copies, gradients, states
        n = sum(a * b for a, b in _adapter_shapes(case))
        return {"bytes": n * (30 if case["bits"] == 32 else 18) + (n // 32 if case["bits"] == 8 else 0), "flops": 15 * n}
    T, H = case["T"], case["H"]
    n = T * H
    if op == "norm_fwd":
        b = 2 + (4 if case["res"] else 0) + (2 if case["y16"] else 0) + (1 if case["rows8"] else 0)
        return {"bytes": n * b + (n // BLOCK if case["rows8"] else 0) + 4 * (T + H), "flops": 6 * n}
    if op == "norm_bwd":
        return {"bytes": n * (8 if case["dres"] else 6) + 4 * (T + H) + (4 * H if case["dw"] else 0), "flops": 10 * n}
    V = case["V"]
    weight = {"bf16": 2 * V * H, "nf4": V * H // 2 + V * H // 64 + 4 * (V * H // 16384),
              "fp8": V * H + V * H // (BLOCK * BLOCK)}[case["W"]]
    return {"bytes": weight + 2 * n * (2 if case["grad"] else 1) + 20 * T, "flops": (4 if case["grad"] else 2) * T * V * H}


# ------------------------------------------------------------------ the definitions in 64 bits
def _two_64(e):
    """2^e in 64 bits, from its bits."""
    return ((e.long() + 1023) << 52).view(torch.float64)


def _step_64(x):
    """The distance of 8-bit values at |x| (64 bits)."""
    _, p = torch.frexp(x)
    return _two_64((p - 1).clamp_min(-6) - 3)


def _scale_64(a):
    """e of the blocks' largest magnitudes, by trying: start below and double while 448 is passed."""
    e = torch.floor(torch.log2(a.clamp_min(2.0 ** -140) / E4M3_MAX)) - 1
    for _ in range(3):
        e = torch.where(a > E4M3_MAX * _two_64(e), e + 1, e)
    return torch.where(a > 0, e.clamp_min(-127), torch.full_like(e, -127))


def _exact_norm_fwd(st):
    h = st["x"].double()
    h = h if st["r"] is None else h + st["r"].double()
    out = {"h": h} if st["r"] is not None else {}
    h = h.to(torch.bfloat16).double()  # the stream is 16-bit by definition
    rstd = (h.pow(2).sum(1) / st["H"] + NORM_EPS).pow(-0.5)
    y = h * rstd.view(-1, 1) * st["w"].double()
    out["rstd"] = rstd
    if st["y16"]:
        out["y"] = y
    if st["rows8"]:  # of the 16-bit y, by definition
        T, H = y.shape
        y = y.to(torch.bfloat16).double()
        G = -(-H // 512)
        codes = torch.zeros((T, -(-H // BLOCK) * BLOCK), dtype=torch.float64, device=y.device)
        scales = torch.full((G, T, 4), 2.0 ** -127, dtype=torch.float64, device=y.device)
        for k in range(0, H, BLOCK):
            piece = y[:, k:k + BLOCK]
            f = _two_64(_scale_64(piece.abs().amax(1)))
            z = piece / f[:, None]
            codes[:, k:k + piece.shape[1]] = torch.round(z / _step_64(z)) * _step_64(z)
            scales[k // 512, :, k // BLOCK % 4] = f
        out["codes"], out["scales"] = codes, scales
    return out


def _exact_head(st):
    V, H = st["V"], st["H"]
    if st["W16"] is not None:
        W = st["W16"].double()
    elif st["W8"] is not None:
        c = st["W8"]["codes"].long()
        ex, fr = (c >> 3) & 15, (c & 7).double()
        W = torch.where(ex == 0, fr * 2.0 ** -9, (1 + fr / 8) * _two_64(ex - 7))
        W = torch.where(c >= 128, -W, W)
        f = _two_64(st["W8"]["scales"].long() - 127)
        for i in range(f.shape[0]):
            W[i * BLOCK:(i + 1) * BLOCK] *= f[i].repeat_interleave(BLOCK)[:H]
    else:
        w = st["W4"]
        W = torch.empty((V, H), dtype=torch.float64, device="cuda")
        table = torch.tensor(NF4_LEVELS, device="cuda")
        for a in range(0, V, 4096):
            b = min(V, a + 4096)
            byte = w["codes"][a * H // 2:b * H // 2].long()
            code = torch.empty((b - a) * H, dtype=torch.int64, device="cuda")
            code[0::2], code[1::2] = byte % 16, byte // 16
            blk = torch.arange(a * H // NF4_BLOCK, b * H // NF4_BLOCK, device="cuda")
            s = (w["q"][blk].float() / 255.0) * w["scale"][blk // NF4_GROUP]  # the format's own fp32 steps
            W[a:b] = (table[code].view(-1, NF4_BLOCK) * s[:, None]).to(torch.bfloat16).double().view(b - a, H)
    loss, lse, dX = [], [], []
    for t in range(0, st["T"], 512):
        X, y, g = st["X"][t:t + 512].double(), st["labels"][t:t + 512], st["dloss"][t:t + 512].double()
        l = X @ W.t()
        has = (y >= 0) & (y < V)
        at = y.clamp(0, V - 1)
        rows = torch.arange(len(y), device=y.device)
        z = torch.logsumexp(l, 1)
        lse.append(z)
        loss.append(torch.where(has, z - l[rows, at], torch.zeros_like(z)))
        if st["grad"]:
            g = torch.where(has, g, torch.zeros_like(g))
            dX.append(g[:, None] * (torch.exp(l - z[:, None]) @ W - W[at]))
    out = {"loss": torch.cat(loss), "lse": torch.cat(lse)}
    if st["grad"]:
        out["dX"] = torch.cat(dX)
    return out


def _hash_bytes(N, seed):
    """Four bytes for each of N / 2 pairs, by 32-bit arithmetic on the host."""
    def mix(x):
        x = (x ^ (x >> np.uint32(16))) * np.uint32(0x85ebca6b)
        x = (x ^ (x >> np.uint32(13))) * np.uint32(0xc2b2ae35)
        return x ^ (x >> np.uint32(16))
    key = mix(np.array([seed], dtype=np.uint32))
    h = mix(np.arange(N // 2, dtype=np.uint32) ^ key)
    return torch.from_numpy(h.astype("<u4").view(np.uint8).copy()).cuda().view(N, 2)  # (for m, for v) of each value


def _exact_adamw(st):
    g = st["grad"].double() * (1.0 if st["scale"] is None else st["scale"].double())
    if st["bits"] == 32:
        m, v = st["m"].double(), st["v"].double()
    else:
        m, v = (st[k].view(torch.float8_e4m3fn).double().view(-1, BLOCK) * _two_64(st[k + "_scales"].long() - 127)[:, None]
                for k in ("m", "v"))
        m, v = m.view(-1), v.view(-1) ** 2
    m = m + (1 - BETA1) * (g - m)
    v = v + (1 - BETA2) * (g ** 2 - v)
    hat_m, hat_v = m / (1 - BETA1 ** st["t"]), v / (1 - BETA2 ** st["t"])
    p = st["master"].double()
    p = p * (1 - RATE * DECAY) - RATE * hat_m / (hat_v.sqrt() + ADAM_EPS)
    out = {"param": p, "master": p}
    if st["bits"] == 32:
        return {**out, "m": m, "v": v}
    u = (_hash_bytes(st["N"], st["seed"]).double() + 0.5) / 256
    for k, (name, x) in enumerate((("m", m), ("v", v.sqrt()))):
        b = x.view(-1, BLOCK)
        f = _two_64(_scale_64(b.abs().amax(1)))
        z = b / f[:, None]
        n = torch.floor(z.abs() / _step_64(z) + u[:, k].view(-1, BLOCK))
        n = torch.where(z != 0, n.clamp_min(1), n) if name == "v" else n
        out[name] = (torch.sign(z) * n * _step_64(z)).view(-1)
        out[name + "_scales"] = f
    return out


def exact(case, seed):
    st = prepare(case, seed)
    op = case["op"]
    if op == "norm_fwd":
        return _exact_norm_fwd(st)
    if op == "norm_bwd":
        h, dy, rstd, w = st["h"].double(), st["dy"].double(), st["rstd"].double(), st["w"].double()
        inner = (dy * w * h).sum(1) / st["H"]
        dh = (dy * w) * rstd[:, None] - h * (inner * rstd ** 3)[:, None]
        out = {"dh": dh if st["dr"] is None else dh + st["dr"].double()}
        if st["dw"]:
            out["dw"] = (dy * h).t() @ rstd
        return out
    return _exact_head(st) if op == "head" else _exact_adamw(st)
