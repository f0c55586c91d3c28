"""Measured cases of the operators around the sketched linear layer in a fine-tuning step.

Three operators:

* ``norm``: layer norm or RMS norm of [T, d] rows, forward alone (serving), forward and
  backward (training), or forward with the 8-bit checkpoint of its output;
* ``lut8``: the 8-bit checkpoint of a layer's input and the LUT gradient that reads it;
* ``loss``: the head product, softmax cross entropy over the vocabulary and its
  gradients for the hidden states and (for a trained head) the head's weight.

``run`` computes the plain form in elementary torch operations, or calls the package when
``own`` is true; ``exact`` computes the definition in 64 bits.
"""
import math

import torch

own = False

IGNORE = -100
DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}


# ---------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------

def listed():
    return [
        # the norm in front of a projection while serving one token, 70B width
        dict(name="norm_token", op="norm", T=1, d=8192, dtype="bf16", wtype="bf16", rms=True, what="fwd"),
        # the norms of a 7B fine-tuning step with trained fp32 weights
        dict(name="norm_train_7b", op="norm", T=8192, d=4096, dtype="bf16", wtype="fp32", rms=False, what="train"),
        # a small model in fp32, rows of odd length
        dict(name="norm_train_odd", op="norm", T=1111, d=1001, dtype="fp32", wtype="fp32", rms=False, what="train"),
        # the norm in front of the 13B projections, with the checkpoint they keep for their backward pass
        dict(name="norm_ckpt_13b", op="norm", T=4096, d=5120, dtype="bf16", wtype="bf16", rms=True, what="ckpt"),
        # one layer of a small model, a short batch
        dict(name="lut8_few", op="lut8", T=33, n=256, d=512, bits=3, gpr=4, sets=1),
        # gate_proj of the 7B fine-tuning step
        dict(name="lut8_gate_7b", op="lut8", T=8192, n=11008, d=4096, bits=2, gpr=8, sets=1),
        # q_proj of a 13B training step whose tokens belong to eight tasks
        dict(name="lut8_sets_13b", op="lut8", T=4096, n=5120, d=5120, bits=4, gpr=4, sets=8),
        # scoring a few tokens: per-token losses, no gradient
        dict(name="loss_score", op="loss", T=16, V=32000, d=4096, reduction="none", what="loss", ignored=0.0),
        # a 7B fine-tuning step with a frozen head
        dict(name="loss_frozen_7b", op="loss", T=4096, V=32000, d=4096, reduction="mean", what="dh", ignored=0.0),
        # the same with a trained head
        dict(name="loss_full_7b", op="loss", T=8192, V=32000, d=4096, reduction="mean", what="dhdw", ignored=0.0),
        # a padded batch of 13B width over an odd vocabulary
        dict(name="loss_odd_13b", op="loss", T=1029, V=50021, d=5120, reduction="sum", what="dh", ignored=0.3),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["norm", "lut8", "loss"])
    if op == "norm":
        what = rng.choice(["fwd", "train", "ckpt"])
        dtype = "bf16" if what == "ckpt" else rng.choice(["bf16", "fp16", "fp32"])
        T = _log_int(rng, 1, 16384)
        d = _log_int(rng, 64, min(16384, max(64, (1 << 25) // T)))
        if what == "ckpt":
            d = (d + 31) // 32 * 32
        return dict(op=op, T=T, d=d, dtype=dtype, wtype=rng.choice([dtype, "fp32"]), rms=rng.random() < 0.5, what=what)
    if op == "lut8":
        gpr = rng.choice([1, 2, 3, 4, 8])
        return dict(op=op, T=_log_int(rng, 1, 8192), n=8 * _log_int(rng, 4, 1024),
                    d=32 * gpr * max(1, _log_int(rng, 4, 160) // gpr), bits=rng.choice([2, 3, 4]), gpr=gpr,
                    sets=rng.choice([1, 1, 3, 8]))
    what = rng.choice(["loss", "dh", "dhdw"])
    T, d = _log_int(rng, 1, 8192), 8 * _log_int(rng, 16, 640)
    return dict(op=op, T=T, V=_log_int(rng, 1000, min(64000, (1 << 40) // (T * d))), d=d,
                reduction=rng.choice(["mean", "sum"]) if what != "loss" else rng.choice(["none", "mean"]), what=what,
                ignored=rng.choice([0.0, 0.1, 0.5]))


def work(case):
    T = case["T"]
    if case["op"] == "norm":
        d, e = case["d"], DTYPES[case["dtype"]].itemsize
        w = d * DTYPES[case["wtype"]].itemsize * (1 if case["rms"] else 2)
        rows = T * d * e
        if case["what"] == "fwd":
            return {"bytes": 2 * rows + w, "flops": 8 * T * d}
        if case["what"] == "ckpt":      # y, and its checkpoint read back
            return {"bytes": 3 * rows + w + T * d // 32 * 33, "flops": 12 * T * d}
        return {"bytes": 4 * rows + 2 * w, "flops": 20 * T * d}    # x and dy read, y and dx written
    if case["op"] == "lut8":
        n, d = case["n"], case["d"]
        bins = 4 * case["sets"] * n * case["gpr"] * (1 << case["bits"])
        return {"bytes": 2 * T * d + 2 * T * n + n * _row_bytes(d, case["bits"]) + bins, "flops": 2 * T * n * d}
    V, d = case["V"], case["d"]
    products = {"loss": 1, "dh": 2, "dhdw": 3}[case["what"]]
    b = 2 * T * d + 2 * V * d + 12 * T
    if case["what"] != "loss":
        b += 2 * T * d
    if case["what"] == "dhdw":
        b += 2 * V * d
    return {"bytes": b, "flops": 2 * products * T * V * d}


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------

def _row_bytes(d, bits):
    return ((d * bits + 7) // 8 + 15) // 16 * 16


def _pack(idx, bits):
    """uint8 [n, d] -> packed rows: 4-bit two per byte (low nibble first), 2-bit four per
    byte, 3-bit 32 indices in three little-endian 32-bit words; rows padded to 16 bytes."""
    n, d = idx.shape
    per = 8 if bits == 3 else 8 // bits                       # indices per group of whole bytes
    v = idx.view(n, d // per, per).to(torch.int32)
    word = (v << (torch.arange(per, device=idx.device, dtype=torch.int32) * bits)).sum(-1)
    nb = per * bits // 8
    b = (word[..., None] >> (8 * torch.arange(nb, device=idx.device, dtype=torch.int32))) & 255
    out = torch.zeros((n, _row_bytes(d, bits)), dtype=torch.uint8, device=idx.device)
    out[:, : d * bits // 8] = b.reshape(n, -1).to(torch.uint8)
    return out


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed * 2654435761 % (1 << 62))
    dev = "cuda"

    def normal(*shape):
        return torch.randn(*shape, device=dev, generator=g)

    T = case["T"]
    s = dict(case)
    if case["op"] in ("norm", "lut8"):
        d = case["d"]
        # a residual stream: some channels are much larger than the rest, rows differ in size
        gain = torch.exp(0.5 * normal(d)) * (1 + 12 * (torch.rand(d, device=dev, generator=g) < 0.01))
        x = normal(T, d) * gain * torch.exp(0.3 * normal(T, 1)) + 0.1 * normal(d)
    if case["op"] == "norm":
        dt, wt = DTYPES[case["dtype"]], DTYPES[case["wtype"]]
        s["x"] = x.to(dt)
        s["w"] = (1 + 0.2 * normal(d)).to(wt)
        s["b"] = None if case["rms"] else (0.1 * normal(d)).to(wt)
        s["eps"] = 1e-5
        s["dy"] = normal(T, d).to(dt) if case["what"] == "train" else None
    elif case["op"] == "lut8":
        n, bits = case["n"], case["bits"]
        s["x"] = x.to(torch.bfloat16)
        s["dy"] = (1e-2 * normal(T, n)).to(torch.bfloat16)
        s["idx"] = torch.randint(0, 1 << bits, (n, d), device=dev, generator=g, dtype=torch.uint8)
        s["packed"] = _pack(s["idx"], bits)
        s["task"] = (torch.randint(0, case["sets"], (T,), device=dev, generator=g, dtype=torch.int32)
                     if case["sets"] > 1 else None)
    else:
        V, d = case["V"], case["d"]
        s["w"] = (normal(V, d) / math.sqrt(d)).to(torch.bfloat16)
        y = torch.randint(0, V, (T,), device=dev, generator=g)
        # hidden states that lean towards their target by different amounts: some tokens
        # are predicted surely, some not at all
        lean = 14 * torch.rand(T, 1, device=dev, generator=g)
        s["h"] = (1.5 * normal(T, d) + lean * s["w"][y].float()).to(torch.bfloat16)
        s["y"] = torch.where(torch.rand(T, device=dev, generator=g) < case["ignored"], IGNORE, y)
        if case["what"] != "loss":
            s["h"].requires_grad_()
        if case["what"] == "dhdw":
            s["w"].requires_grad_()
    return s


# ---------------------------------------------------------------------------
# plain forms (32 bits) and the package's calls
# ---------------------------------------------------------------------------

def _checkpoint(x):
    """fp32 values that the 8-bit checkpoint of x stands for: blocks of 32 columns, scale 2^e
    with e the least integer for which max|x| <= 127 * 2^e (at most 121, at least -126)."""
    T, d = x.shape
    v = x.float().view(T, d // 32, 32)
    m, ex = torch.frexp(v.abs().amax(-1, keepdim=True))       # amax = m * 2^ex, m in [0.5, 1)
    e = (ex - 7 + (m > 127 / 128).to(ex.dtype)).clamp(-126, 121)
    q = torch.round(torch.ldexp(v, -e)).clamp(-127, 127)
    return torch.ldexp(q, e).view(T, d)


def _norm_plain(s):
    x, w = s["x"].float(), s["w"].float()
    mu = 0.0 if s["rms"] else x.mean(1, keepdim=True)
    c = x - mu
    r = torch.rsqrt((c * c).mean(1, keepdim=True) + s["eps"])
    xh = c * r
    y = xh * w if s["b"] is None else xh * w + s["b"].float()
    out = {"y": y.to(s["x"].dtype)}
    if s["what"] == "ckpt":
        out["checkpoint"] = _checkpoint(out["y"]).to(s["x"].dtype)
    if s["what"] == "train":
        dy = s["dy"].float()
        gw = dy * w
        m1 = 0.0 if s["rms"] else gw.mean(1, keepdim=True)
        dx = r * (gw - m1 - xh * (gw * xh).mean(1, keepdim=True))
        out["dx"] = dx.to(s["x"].dtype)
        out["dw"] = (dy * xh).sum(0).to(s["w"].dtype)
        if s["b"] is not None:
            out["db"] = dy.sum(0).to(s["b"].dtype)
    return out


def _norm_own(s):
    from compressive_fine_tuning_b200 import sk
    if s["what"] == "fwd":
        return {"y": sk.layer_norm(s["x"], s["w"], s["b"], s["eps"], s["rms"])}
    y, mean, rstd, ck = sk.layer_norm_fwd(s["x"], s["w"], s["b"], s["eps"], s["rms"], ckpt=s["what"] == "ckpt")
    out = {"y": y}
    if s["what"] == "ckpt":
        out["checkpoint"] = sk.ckpt8_dequant(ck)
    else:
        out["dx"], out["dw"], db = sk.layer_norm_bwd(s["dy"], s["x"], s["w"], mean, rstd, s["rms"],
                                                     bias=s["b"] is not None)
        if s["b"] is not None:
            out["db"] = db
    return out


def _lut8_plain(s):
    n, d, gpr, k = s["n"], s["d"], s["gpr"], 1 << s["bits"]
    x, dy = _checkpoint(s["x"]), s["dy"].float()
    if s["task"] is not None:
        mine = s["task"][None, :, None] == torch.arange(s["sets"], device=dy.device)[:, None, None]
        dy = dy * mine                                          # [sets, T, n]
    else:
        dy = dy[None]
    G = dy.transpose(1, 2) @ x                                  # [sets, n, d]
    idx = s["idx"].long().view(1, n, gpr, d // gpr).expand(s["sets"], n, gpr, d // gpr)
    out = torch.zeros((s["sets"], n, gpr, k), device=G.device)
    return {"dlut": out.scatter_add_(3, idx, G.view(s["sets"], n, gpr, d // gpr))}


def _lut8_own(s):
    from compressive_fine_tuning_b200 import sk
    ck = sk.ckpt8(s["x"])
    return {"dlut": sk.linear_bwd_lut_ckpt8(s["packed"], s["bits"], s["gpr"], ck, s["dy"], s["task"], s["sets"])}


def _loss_plain(s):
    h, w, y = s["h"].detach().float(), s["w"].detach().float(), s["y"]
    valid = y != IGNORE
    safe = torch.where(valid, y, 0)
    logits = h @ w.t()
    m = logits.amax(1, keepdim=True)
    lse = m + torch.log(torch.exp(logits - m).sum(1, keepdim=True))
    losses = torch.where(valid, (lse - logits.gather(1, safe[:, None]))[:, 0], 0.0)
    if s["reduction"] == "none":
        return {"loss": losses}
    c = valid.float() / valid.sum().clamp(min=1) if s["reduction"] == "mean" else valid.float()
    out = {"loss": (losses * c).sum()}
    if s["what"] != "loss":
        dl = torch.exp(logits - lse)
        dl[torch.arange(len(y), device=y.device), safe] -= 1.0
        dl *= c[:, None]
        out["dh"] = (dl @ w).to(torch.bfloat16)
        if s["what"] == "dhdw":
            out["dw"] = (dl.t() @ h).to(torch.bfloat16)
    return out


def _loss_own(s):
    from compressive_fine_tuning_b200 import sk
    loss = sk.linear_cross_entropy(s["h"], s["w"], s["y"], ignore_index=IGNORE, reduction=s["reduction"])
    out = {"loss": loss.detach()}
    if s["what"] == "dh":
        out["dh"], = torch.autograd.grad(loss, [s["h"]])
    elif s["what"] == "dhdw":
        out["dh"], out["dw"] = torch.autograd.grad(loss, [s["h"], s["w"]])
    return out


def run(s):
    if own:
        return {"norm": _norm_own, "lut8": _lut8_own, "loss": _loss_own}[s["op"]](s)
    with torch.no_grad():
        return {"norm": _norm_plain, "lut8": _lut8_plain, "loss": _loss_plain}[s["op"]](s)


# ---------------------------------------------------------------------------
# the definitions in 64 bits
# ---------------------------------------------------------------------------

def _checkpoint64(v):
    """Nearest multiple of 2^e (ties to the even multiple) for every value of a block of 32."""
    b = v.double().reshape(v.shape[0], -1, 32)
    top = b.abs().max(dim=2, keepdim=True).values
    e = torch.ceil(torch.log2(top.clamp(min=1e-300) / 127)).clamp(-126, 121)
    e = torch.where(127 * torch.exp2(e - 1) >= top, (e - 1).clamp(min=-126), e)      # log2 next to a whole number
    e = torch.where(127 * torch.exp2(e) < top, (e + 1).clamp(max=121), e)
    step = torch.exp2(e)
    return ((b / step).round().clamp(-127, 127) * step).reshape(v.shape)


def exact(case, seed):
    s = prepare(case, seed)
    with torch.no_grad():
        if case["op"] == "norm":
            x, w = s["x"].double(), s["w"].double()
            n = x.shape[1]
            mu = torch.zeros_like(x[:, :1]) if s["rms"] else x.sum(1, keepdim=True) / n
            sd = torch.sqrt(((x - mu) ** 2).sum(1, keepdim=True) / n + s["eps"])
            z = (x - mu) / sd
            y = z * w + (0.0 if s["b"] is None else s["b"].double())
            out = {"y": y}
            if s["what"] == "ckpt":
                out["checkpoint"] = _checkpoint64(y.to(s["x"].dtype))
            if s["what"] == "train":
                dy = s["dy"].double()
                u = dy * w
                dx = u - z * ((u * z).sum(1, keepdim=True) / n)
                if not s["rms"]:
                    dx = dx - u.sum(1, keepdim=True) / n
                out["dx"] = dx / sd
                out["dw"] = torch.einsum("td,td->d", dy, z)
                if s["b"] is not None:
                    out["db"] = dy.sum(0)
            return out
        if case["op"] == "lut8":
            x, dy = _checkpoint64(s["x"]), s["dy"].double()
            sets = []
            for tau in range(s["sets"]):
                rows = slice(None) if s["task"] is None else s["task"] == tau
                G = dy[rows].t() @ x[rows]
                G = G.reshape(s["n"], s["gpr"], -1)
                at = s["idx"].reshape(G.shape)
                sets.append(torch.stack([(G * (at == c)).sum(2) for c in range(1 << s["bits"])], dim=2))
            return {"dlut": torch.stack(sets)}
        h, w, y = s["h"].detach().double(), s["w"].detach().double(), s["y"]
        keep = y != IGNORE
        count = max(1, int(keep.sum()))
        scale = 1.0 / count if s["reduction"] == "mean" else 1.0
        losses = torch.zeros(len(y), dtype=torch.float64, device=y.device)
        dh = torch.zeros_like(h)
        dw = torch.zeros_like(w) if s["what"] == "dhdw" else None
        for a in range(0, len(y), 2048):                       # tokens in pieces: 64-bit logits are large
            k = torch.nonzero(keep[a:a + 2048])[:, 0] + a
            z = h[k] @ w.t()
            rows = torch.arange(len(k), device=y.device)
            losses[k] = torch.logsumexp(z, 1) - z[rows, y[k]]
            if s["what"] == "loss":
                continue
            p = torch.softmax(z, 1)
            t = p[rows, y[k]].clone()
            p[rows, y[k]] = 0.0
            p[rows, y[k]] = -torch.where(t < 0.5, 1 - t, p.sum(1))      # 1 - p_target without cancellation
            p *= scale
            dh[k] = p @ w
            if dw is not None:
                dw += p.t() @ h[k]
        if s["reduction"] == "none":
            return {"loss": losses}
        out = {"loss": losses.sum() * scale}
        if s["what"] != "loss":
            out["dh"] = dh
        if dw is not None:
            out["dw"] = dw
        return out
