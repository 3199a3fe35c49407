"""Timed cases of the sublayer operators around the kept tokens: norms before
and after a sublayer, 8-bit activation checkpoints and what the backward pass
computes from them.

``listed()`` and ``draw()`` give the cases, ``prepare()`` the tensors that a
training or decoding program holds before the call, ``run()`` one pass.  With
``own`` false a pass is elementary torch arithmetic in 32 bits, each result
rounded once; with ``own`` true it is the library's calls.  ``exact()`` is the
definition in 64 bits.
"""

import math

import torch

own = False

NORMS = {"none": 0, "rms": 1, "layer": 2}
FORMATS = {"e4m3": 0, "int8": 1}
GROUP = 32       # columns that share one scale of a checkpoint
PAD = 128        # kept rows are padded with zero rows to a multiple of this
BLOCK = 64       # token block of the selection


# --------------------------------------------------------------------- cases
def listed():
    return [
        # one token of one sequence: what a decoding step calls before a sublayer
        dict(name="prenorm-token", op="prenorm", norm="rms", L=1, d=4096, keep=1.0, source="x",
             train=False),
        # LayerNorm with a bias, odd width and length, gradient from the bf16 rows
        dict(name="prenorm-layer-odd", op="prenorm", norm="layer", L=5003, d=1000, keep=0.7,
             source="x", train=True),
        # a layer of the 16384-token workload, half of the tokens kept, gradient from the checkpoint
        dict(name="prenorm-rms-16k", op="prenorm", norm="rms", L=16384, d=4096, keep=0.5,
             source="e4m3", train=True),
        # the small workload's residual stream, per-channel gate, gradient from an int8 checkpoint
        dict(name="postnorm-layer-1k", op="postnorm", norm="layer", L=1024, d=512, keep=0.5,
             source="int8", gate="channel", train=True),
        # a layer of the 32768-token workload, one gate per token and channel
        dict(name="postnorm-rms-32k", op="postnorm", norm="rms", L=32768, d=5120, keep=0.5,
             source="y", gate="token", train=True),
        # a short odd batch saved through its kept ids
        dict(name="checkpoint-int8-odd", op="checkpoint", fmt="int8", L=777, d=648, keep=0.5),
        # every row of a layer's activations saved and brought back
        dict(name="checkpoint-e4m3-16k", op="checkpoint", fmt="e4m3", L=16384, d=4096, keep=1.0),
        # the gated MLP of one token block
        dict(name="gated-block", op="gated", fmt="int8", K=64, d=11008),
        # the gated MLP of the 16384-token workload at half of the tokens
        dict(name="gated-16k", op="gated", fmt="e4m3", K=8192, d=11008),
        # weight gradient of a small projection over a few ragged rows
        dict(name="wgrad-small", op="wgrad", fmt="int8", K=333, n=520, d=512),
        # query projection at the 30 % layer of the 16384-token workload
        dict(name="wgrad-attention-16k", op="wgrad", fmt="int8", K=4928, n=4096, d=4096),
        # down projection of the gated MLP at half of the tokens
        dict(name="wgrad-down-16k", op="wgrad", fmt="e4m3", K=8192, n=4096, d=11008),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["prenorm", "postnorm", "checkpoint", "gated", "wgrad"])
    fmt = rng.choice(["e4m3", "int8"])
    d = 8 * _log(rng, 8, 1024)
    if op == "gated":
        d = 8 * _log(rng, 16, 1376)
        return dict(op=op, fmt=fmt, K=_log(rng, 1, 8192), d=d)
    if op == "wgrad":
        return dict(op=op, fmt=fmt, K=_log(rng, 1, 8192), n=8 * _log(rng, 8, 512), d=d)
    L = min(_log(rng, 1, 32768), (32768 * 5120) // d)
    c = dict(op=op, L=L, d=d, keep=rng.choice([0.3, 0.5, 0.7, 1.0]))
    if op == "checkpoint":
        return dict(c, fmt=fmt)
    c["norm"] = rng.choice(["rms", "layer"] if op == "prenorm" else ["none", "rms", "layer"])
    c["source"] = rng.choice(["x" if op == "prenorm" else "y", fmt])
    c["train"] = rng.random() < 0.8
    if op == "postnorm":
        c["gate"] = rng.choice(["none", "channel", "token"])
    return c


def _blocks(case):
    nb = -(-case["L"] // BLOCK)
    return nb, max(1, int(round(case["keep"] * nb)))


def _kept(case):
    """Kept rows: whole blocks, the (short) last one always among them."""
    if "K" in case:
        return case["K"]
    nb, k = _blocks(case)
    return (k - 1) * BLOCK + case["L"] - (nb - 1) * BLOCK


# --------------------------------------------------------------------- inputs
def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    bf, f32, u8, dev = torch.bfloat16, torch.float32, torch.uint8, "cuda"

    def normal(*shape, scale=1.0, add=0.0):
        return torch.randn(*shape, generator=g, device=dev).mul_(scale).add_(add).to(bf)

    def salient(rows, cols):  # one row in ten carries four times the magnitude
        t = torch.randn(rows, cols, generator=g, device=dev)
        t[torch.rand(rows, generator=g, device=dev) < 0.1] *= 4.0
        return t.to(bf)

    op, d, K = case["op"], case["d"], _kept(case)
    Kp = -(-K // PAD) * PAD
    ld = -(-d // 16) * 16
    s = dict(case=dict(case), K=K, Kp=Kp, K_d=torch.tensor([K], dtype=torch.int32, device=dev))

    def checkpoint(tag):
        s["data" + tag] = torch.zeros(Kp, ld, dtype=u8, device=dev)
        s["scales" + tag] = torch.zeros(Kp, -(-d // (4 * GROUP)) * 4, dtype=u8, device=dev)

    if "L" in case:
        nb, k = _blocks(case)
        pick = torch.randperm(nb - 1, generator=g, device=dev)[: k - 1] if nb > 1 else None
        mask = torch.zeros(nb, dtype=torch.bool, device=dev)
        mask[-1] = True
        if pick is not None:
            mask[pick] = True
        rows = torch.arange(case["L"], device=dev)
        s["idx"] = rows[mask[rows // BLOCK]].to(torch.int32)
        s["rows"] = s["idx"].long()
    if op in ("prenorm", "postnorm"):
        norm, L = case["norm"], case["L"]
        s["x"] = salient(L, d)
        s["w"] = normal(d, scale=0.1, add=1.0) if norm != "none" else None
        s["b"] = normal(d, scale=0.1) if norm == "layer" else None
        s["y"] = torch.zeros(Kp, d, dtype=bf, device=dev) if op == "prenorm" else normal(Kp, d)
        s["stats"] = torch.zeros(Kp, 2, dtype=f32, device=dev) if norm != "none" else None
        s["ws"] = torch.empty(64 << 20, dtype=u8, device=dev)
        if case["source"] in FORMATS:
            checkpoint("")
        if op == "postnorm":
            gate = case["gate"]
            s["gate"] = (None if gate == "none" else
                         normal(d, scale=0.1, add=0.5) if gate == "channel" else
                         torch.rand(Kp, d, generator=g, device=dev).to(bf))
            s["scale"] = 0.5
        if case["train"]:
            s["dx"] = normal(L, d, scale=0.01)
            if norm != "none":
                s["dw"] = torch.zeros(d, dtype=f32, device=dev)
            if norm == "layer":
                s["db"] = torch.zeros(d, dtype=f32, device=dev)
            if op == "prenorm":
                s["dy"] = normal(Kp, d, scale=0.01)
            else:
                s["dy"] = torch.zeros(Kp, d, dtype=bf, device=dev)
                if case["gate"] == "channel":
                    s["dgate"] = torch.zeros(d, dtype=f32, device=dev)
                elif case["gate"] == "token":
                    s["dgate"] = torch.zeros(Kp, d, dtype=bf, device=dev)
    elif op == "checkpoint":
        s["x"] = salient(case["L"], d)
        s["y"] = torch.zeros(Kp, d, dtype=bf, device=dev)
        checkpoint("")
    elif op == "gated":
        s["gate"], s["up"] = salient(Kp, d), salient(Kp, d)
        s["da"] = normal(Kp, d, scale=0.01)
        for n in ("a", "a_again", "dgate", "dup"):
            s[n] = torch.zeros(Kp, d, dtype=bf, device=dev)
        checkpoint("_gate")
        checkpoint("_up")
    else:
        x = salient(Kp, d)
        checkpoint("")
        q, e = _quantise(x[:K], case["fmt"])
        s["data"][:K, :d] = q
        s["scales"][:K, : e.shape[1]] = e
        s["dy"] = normal(Kp, case["n"], scale=0.01)
        s["dw"] = torch.zeros(case["n"], d, dtype=f32, device=dev)
    return s


# --------------------------------------------------------------------- plain forms
def _groups(v):
    """[K, d] -> [K, groups, 32], the last group filled up with zeros."""
    K, d = v.shape
    n = -(-d // GROUP)
    return torch.nn.functional.pad(v, (0, n * GROUP - d)).reshape(K, n, GROUP)


def _power(e):
    """2^e as float32 for integers e in [-126, 127], from the exponent's bits."""
    return ((e.to(torch.int32) + 127) << 23).view(torch.float32)


def _quantise(x, fmt):
    """Codes (uint8 [K, d]) and scale codes (uint8 [K, groups]) of bf16 rows.

    The scale of 32 columns is the smallest power of two (code - 127) that
    brings their largest magnitude to at most 448 (e4m3) or 127 (int8)."""
    v = _groups(x.float())
    most = 448.0 if fmt == "e4m3" else 127.0
    m, e = torch.frexp(v.abs().amax(-1) / most)       # amax / most = m 2^e, 1/2 <= m < 1
    e = torch.where(m > 0.5, e, e - 1).clamp(min=-124)
    e = torch.where(m == 0, torch.full_like(e, -124), e)
    half = e // 2                                     # 2^-e in two factors
    t = v * _power(-half)[..., None] * _power(half - e)[..., None]
    t = t.reshape(x.shape[0], -1)[:, : x.shape[1]].contiguous()
    q = t.to(torch.float8_e4m3fn) if fmt == "e4m3" else torch.round(t).to(torch.int8)
    return q.view(torch.uint8), (e + 127).to(torch.uint8)


def _values(q, codes, fmt):
    """float32 values that codes and scale codes stand for."""
    t = q.contiguous().view(torch.float8_e4m3fn if fmt == "e4m3" else torch.int8).float()
    f = _power(codes.to(torch.int32) - 127).repeat_interleave(GROUP, 1)[:, : t.shape[1]]
    return t * f


def _save(s, x, fmt, tag=""):
    q, e = _quantise(x, fmt)
    s["data" + tag][: s["K"], : q.shape[1]] = q
    s["scales" + tag][: s["K"], : e.shape[1]] = e
    return _values(q, e, fmt)


def _statistics(v, norm, eps):
    if norm == "none":
        return torch.zeros_like(v[:, :1]), torch.ones_like(v[:, :1])
    mean = v.mean(1, keepdim=True) if norm == "layer" else torch.zeros_like(v[:, :1])
    return mean, 1.0 / torch.sqrt((v - mean).square().mean(1, keepdim=True) + eps)


def _norm_backward(gxhat, xhat, rstd, norm):
    if norm == "none":
        return gxhat
    g = gxhat - xhat * (gxhat * xhat).mean(1, keepdim=True)
    if norm == "layer":
        g = g - gxhat.mean(1, keepdim=True)
    return g * rstd


EPS = 1e-5


def _plain_prenorm(s):
    c, K, bf = s["case"], s["K"], torch.bfloat16
    w = s["w"].float()
    v = s["x"][s["rows"]].float()
    mean, rstd = _statistics(v, c["norm"], EPS)
    y = (v - mean) * rstd * w
    if s["b"] is not None:
        y = y + s["b"].float()
    s["y"][:K] = y.to(bf)
    s["y"][K:] = 0
    s["stats"][:K] = torch.cat([mean, rstd], 1)
    if c["source"] in FORMATS:
        v = _save(s, s["x"][s["rows"]], c["source"])
    if c["train"]:
        xhat = (v - mean) * rstd
        dy = s["dy"][:K].float()
        dv = _norm_backward(dy * w, xhat, rstd, c["norm"])
        s["dx"][s["rows"]] = (s["dx"][s["rows"]].float() + dv).to(bf)
        s["dw"] += (dy * xhat).sum(0)
        if s["b"] is not None:
            s["db"] += dy.sum(0)


def _plain_postnorm(s):
    c, K, bf = s["case"], s["K"], torch.bfloat16
    v = s["y"][:K].float()
    mean, rstd = _statistics(v, c["norm"], EPS)
    w = s["w"].float() if s["w"] is not None else 1.0
    b = s["b"].float() if s["b"] is not None else 0.0
    gate = 1.0 if s["gate"] is None else s["gate"].float()
    if c["gate"] == "token":
        gate = gate[:K]
    n = (v - mean) * rstd * w + b
    s["x"][s["rows"]] = (s["x"][s["rows"]].float() + s["scale"] * (gate * n)).to(bf)
    if s["stats"] is not None:
        s["stats"][:K] = torch.cat([mean, rstd], 1)
    if c["source"] in FORMATS:
        v = _save(s, s["y"][:K], c["source"])
    if c["train"]:
        vhat = (v - mean) * rstd
        dz = s["scale"] * s["dx"][s["rows"]].float()
        dn = dz * gate
        s["dy"][:K] = _norm_backward(dn * w, vhat, rstd, c["norm"]).to(bf)
        s["dy"][K:] = 0
        if c["norm"] != "none":
            s["dw"] += (dn * vhat).sum(0)
        if c["norm"] == "layer":
            s["db"] += dn.sum(0)
        if c["gate"] == "channel":
            s["dgate"] += (dz * (vhat * w + b)).sum(0)
        elif c["gate"] == "token":
            s["dgate"][:K] = (dz * (vhat * w + b)).to(bf)


def _plain_checkpoint(s):
    s["y"][: s["K"]] = _save(s, s["x"][s["rows"]], s["case"]["fmt"]).to(torch.bfloat16)
    s["y"][s["K"]:] = 0


def _plain_gated(s):
    K, bf, fmt = s["K"], torch.bfloat16, s["case"]["fmt"]
    g, u = s["gate"][:K], s["up"][:K]
    s["a"][:K] = (g.float() / (1.0 + torch.exp(-g.float())) * u.float()).to(bf)
    g, u = _save(s, g, fmt, "_gate"), _save(s, u, fmt, "_up")
    sig = 1.0 / (1.0 + torch.exp(-g))
    da = s["da"][:K].float()
    s["a_again"][:K] = (g * sig * u).to(bf)
    s["dup"][:K] = (da * g * sig).to(bf)
    s["dgate"][:K] = (da * u * sig * (1.0 + g * (1.0 - sig))).to(bf)
    for n in ("a", "a_again", "dup", "dgate"):
        s[n][K:] = 0


def _plain_wgrad(s):
    K, d = s["K"], s["case"]["d"]
    x = _values(s["data"][:K, :d], s["scales"][:K, : -(-d // GROUP)], s["case"]["fmt"])
    s["dw"] += s["dy"][:K].float().t() @ x


# --------------------------------------------------------------------- the library's calls
def _own(s):
    from contextual_token_sparsity_b200 import lemo
    c, op, K_d = s["case"], s["case"]["op"], s["K_d"]
    ck = s.get("ck")
    if ck is None:  # the handles that a program makes once, beside its buffers
        fmt = c.get("fmt") or c.get("source")
        ck = s["ck"] = {t: lemo.make_checkpoint(s["data" + t], s["scales" + t], FORMATS[fmt], c["d"])
                        for t in ("", "_gate", "_up") if "data" + t in s}
    if op == "prenorm":
        saved = ck.get("")
        norm = NORMS[c["norm"]]
        lemo.lemo_norm_gather(norm, s["x"], s["w"], s["b"], EPS, s["idx"], K_d, PAD, s["y"],
                              stats=s["stats"], checkpoint=saved)
        if c["train"]:
            lemo.lemo_norm_gather_backward(norm, s["dy"], s["w"], s["stats"], s["idx"], K_d,
                                           s["dx"], s["ws"], x=None if saved else s["x"],
                                           checkpoint=saved, dweight=s["dw"], dbias=s.get("db"))
    elif op == "postnorm":
        saved = ck.get("")
        norm = NORMS[c["norm"]]
        lemo.lemo_norm_scatter(norm, s["x"], s["y"], s["w"], s["b"], EPS, s["gate"], s["scale"],
                               s["idx"], K_d, stats=s["stats"], checkpoint=saved)
        if c["train"]:
            lemo.lemo_norm_scatter_backward(norm, s["dx"], s["w"], s["b"], s["stats"], s["gate"],
                                            s["scale"], s["idx"], K_d, PAD, s["dy"], s["ws"],
                                            y=None if saved else s["y"], checkpoint=saved,
                                            dweight=s.get("dw"), dbias=s.get("db"),
                                            dgate=s.get("dgate"))
    elif op == "checkpoint":
        lemo.lemo_checkpoint_save(s["x"], s["idx"], K_d, ck[""])
        lemo.lemo_checkpoint_restore(ck[""], K_d, PAD, s["y"])
    elif op == "gated":
        lemo.lemo_gated_mlp(s["gate"], s["up"], K_d, PAD, s["a"], ck["_gate"], ck["_up"])
        lemo.lemo_gated_mlp_backward(ck["_gate"], ck["_up"], s["da"], K_d, PAD, s["dgate"],
                                     s["dup"], a=s["a_again"])
    else:
        lemo.lemo_checkpoint_weight_grad(ck[""], s["dy"], K_d, s["dw"])


_OUT = {
    "prenorm": ("y", "stats", "dx", "dw", "db"),
    "postnorm": ("x", "stats", "dy", "dw", "db", "dgate"),
    "checkpoint": ("y",),
    "gated": ("a", "a_again", "dgate", "dup"),
    "wgrad": ("dw",),
}


def run(state):
    s, c = state, state["case"]
    if own:
        _own(s)
    else:
        {"prenorm": _plain_prenorm, "postnorm": _plain_postnorm, "checkpoint": _plain_checkpoint,
         "gated": _plain_gated, "wgrad": _plain_wgrad}[c["op"]](s)
    train = c.get("train", True)
    names = [n for n in _OUT[c["op"]] if train or n in ("y", "x", "stats")]
    out = {n: s[n] for n in names if s.get(n) is not None}
    fmt = c.get("fmt") or c.get("source")
    if c["op"] != "wgrad" and fmt in FORMATS:
        kind = torch.float8_e4m3fn if fmt == "e4m3" else torch.int8
        for t in ("", "_gate", "_up"):
            if "data" + t in s:  # the codes as the numbers they are, and the scales' exponents
                out["data" + t] = s["data" + t].view(kind)
                out["scales" + t] = s["scales" + t]
    return out


# --------------------------------------------------------------------- work of one pass
def work(case):
    op, d, K = case["op"], case["d"], _kept(case)
    ck = 1.0 + 1.0 / GROUP              # bytes of one checkpointed value
    if op == "wgrad":
        n = case["n"]
        return dict(bytes=ck * K * d + 2.0 * K * n + 8.0 * n * d, flops=2.0 * K * n * d)
    if op == "checkpoint":
        return dict(bytes=K * d * (2 + ck + 2) + 4 * K, flops=4.0 * K * d)
    if op == "gated":
        return dict(bytes=K * d * (2 + 2 + 2 + 2 * ck + 2 + 2 + 2 + 2), flops=40.0 * K * d)
    saved = ck if case["source"] in FORMATS else 0.0
    per = 2 + 2 + saved                 # prenorm: x read, y written; postnorm: y, x read
    if op == "postnorm":
        per += 2 + (2 if case["gate"] == "token" else 0)        # x written; gate rows read
    if case["train"]:                   # dy and dx read, one of them written
        per += 2 + 2 + (2 if op == "prenorm" else 0)
        if op == "postnorm" and case["gate"] == "token":
            per += 2                    # gradient rows of the gate
    return dict(bytes=K * (d * per + 12.0), flops=30.0 * K * d)


# --------------------------------------------------------------------- the definition in 64 bits
def _two_to(k):
    """2^k in 64 bits, exactly."""
    return ((k.to(torch.int64) + 1023) << 52).view(torch.float64)


def _round_codes(x, fmt):
    """The rows' quantised values in 64 bits, from the definition: magnitudes
    scaled by a power of two and rounded, ties to even, to the format's grid."""
    K, d = x.shape
    out = torch.empty(K, d, dtype=torch.float64, device=x.device)
    most = 448.0 if fmt == "e4m3" else 127.0
    codes = []
    for c in range(0, d, GROUP):
        v = x[:, c: c + GROUP].double()
        peak = v.abs().max(1).values
        k = torch.ceil(torch.log2(torch.clamp(peak, min=2.0 ** -140) / most))
        k = torch.where(peak > most * _two_to(k), k + 1, k)          # log2 next to a power of two
        k = torch.where(peak <= most * _two_to(k - 1), k - 1, k)
        k = torch.clamp(k, min=-124.0)
        codes.append((k + 127).to(torch.uint8))
        t = v / _two_to(k)[:, None]
        if fmt == "int8":
            r = torch.round(t)
        else:
            step = _two_to(torch.clamp(torch.frexp(t).exponent - 1, min=-6) - 3)
            r = torch.round(t / step) * step
        out[:, c: c + GROUP] = r * _two_to(k)[:, None]
    return out, torch.stack(codes, 1)


def _exact_norm(v, norm):
    if norm == "none":
        return torch.zeros(v.shape[0], 1, dtype=v.dtype, device=v.device), torch.ones(v.shape[0], 1, dtype=v.dtype, device=v.device)
    n = v.shape[1]
    mean = v.sum(1, keepdim=True) / n if norm == "layer" else 0.0 * v[:, :1]
    var = ((v - mean) ** 2).sum(1, keepdim=True) / n
    return mean, (var + EPS) ** -0.5


def _exact_dnorm(dn, v, mean, rstd, norm):
    """d/dv of sum(dn * (v - mean) rstd) with the statistics' own dependence on v."""
    if norm == "none":
        return dn
    n, c = v.shape[1], v - mean
    dot = (dn * c).sum(1, keepdim=True)
    out = dn * rstd - c * rstd ** 3 * dot / n
    return out - rstd * dn.sum(1, keepdim=True) / n if norm == "layer" else out


def exact(case, seed):
    s = prepare(case, seed)
    op, K, Kp = case["op"], s["K"], s["Kp"]

    def tall(v):
        return torch.nn.functional.pad(v, (0, 0, 0, Kp - K))

    if op == "wgrad":
        t = s["data"][:K, : case["d"]].contiguous()
        t = t.view(torch.float8_e4m3fn if case["fmt"] == "e4m3" else torch.int8).double()
        e = s["scales"].to(torch.int64) - 127
        for c in range(0, case["d"], GROUP):
            t[:, c: c + GROUP] *= _two_to(e[:K, c // GROUP])[:, None]
        return dict(dw=torch.matmul(s["dy"][:K].double().t(), t))
    if op == "checkpoint":
        return dict(y=tall(_round_codes(s["x"][s["rows"]], case["fmt"])[0]))
    if op == "gated":
        def silu(v):
            return v * torch.sigmoid(v)
        g, u, da = s["gate"][:K], s["up"][:K], s["da"][:K].double()
        out = dict(a=tall(silu(g.double()) * u.double()))
        g, u = _round_codes(g, case["fmt"])[0], _round_codes(u, case["fmt"])[0]
        sg = torch.sigmoid(g)
        out["a_again"] = tall(silu(g) * u)
        out["dgate"] = tall(da * u * (sg + g * sg * (1 - sg)))
        out["dup"] = tall(da * silu(g))
        return out
    norm, rows = case["norm"], s["rows"]
    w = s["w"].double() if s["w"] is not None else torch.ones(case["d"], dtype=torch.float64, device="cuda")
    b = s["b"].double() if s["b"] is not None else 0.0 * w
    raw = s["x"][rows] if op == "prenorm" else s["y"][:K]
    v = raw.double()
    mean, rstd = _exact_norm(v, norm)
    out = {}
    n = (v - mean) * rstd * w + b
    if norm != "none":
        out["stats"] = tall(torch.cat([mean, rstd], 1))
    if op == "prenorm":
        out["y"] = tall(n)
    else:
        gate = 1.0 if s["gate"] is None else s["gate"].double()
        gate = gate[:K] if case["gate"] == "token" else gate
        x = s["x"].double()
        x[rows] += s["scale"] * gate * n
        out["x"] = x
    if case["source"] in FORMATS:
        v = _round_codes(raw, case["source"])[0]
    if not case["train"]:
        return out
    # the backward pass takes the forward pass's statistics with the checkpoint's values
    vhat = (v - mean) * rstd
    n_of = vhat.shape[1]

    def back(g):
        if norm == "none":
            return g
        if case["source"] not in FORMATS:
            return _exact_dnorm(g, v, mean, rstd, norm)
        r = g - vhat * (g * vhat).sum(1, keepdim=True) / n_of
        return rstd * (r - g.sum(1, keepdim=True) / n_of if norm == "layer" else r)

    if op == "prenorm":
        dy = s["dy"][:K].double()
        dx = s["dx"].double()
        dx[rows] += back(dy * w)
        out["dx"] = dx
        out["dw"] = (dy * vhat).sum(0)
        if norm == "layer":
            out["db"] = dy.sum(0)
        return out
    dz = s["scale"] * s["dx"][rows].double()
    out["dy"] = tall(back(dz * gate * w))
    if norm != "none":
        out["dw"] = (dz * gate * vhat).sum(0)
    if norm == "layer":
        out["db"] = (dz * gate).sum(0)
    if case["gate"] == "channel":
        out["dgate"] = (dz * (vhat * w + b)).sum(0)
    elif case["gate"] == "token":
        out["dgate"] = tall(dz * (vhat * w + b))
    return out
