"""The operators around the MoE layer's routed experts, and how they are measured.

A transformer block of this layer is  y = x + dropout(MoE(n) + FFN(n)),
n = layer_norm(x): this file holds the layer norm, the dropout with its
residual sum and the shared (dense) gated feed-forward block, forward and
backward, in their plain form, the calls a user makes of the library for
the same results, and their definition in 64 bits.

  layer norm   y = (x - mean) rstd w + b per row, rstd = 1 / sqrt(var + eps);
               dx = rstd (g - mean(g) - xh mean(g xh)) + addend with g = dy w
               and xh = (x - mean) rstd; dw = sum_t dy xh, db = sum_t dy
  dropout      out = residual + keep * x / (1 - p); element i is kept where
               the 16-bit half i % 2 of word (i % 8) / 2 of the Philox4x32-10
               block with counter (i / 8, offset) and key seed is at least
               thr = round(65536 p); 1 / (1 - p) is 65536 / (65536 - thr)
  gated FFN    H = [x W1 | x W3], A = silu(H1) * H3, y = A W2 + addend; from
               dout: dA = dout W2^T, dH = [dA H3 silu'(H1) | dA silu(H1)],
               dx = dH [W1 | W3]^T + addend, dW1 | dW3 = x^T dH, dW2 = A^T dout
"""
import math

import numpy as np
import torch

#: False: run() computes the plain forms.  True: it calls the library.
own = False

_TYPES = {"f32": torch.float32, "bf16": torch.bfloat16}
_SIZE = {"f32": 4, "bf16": 2}
_EPS = 1e-5


def _ln(direction, T, d, dtype, wtype, addend=False):
    return {"op": "layernorm", "dir": direction, "T": T, "d": d, "dtype": dtype, "wtype": wtype, "addend": addend}


def _dropout(direction, T, d, dtype, p, residual):
    return {"op": "dropout", "dir": direction, "T": T, "d": d, "dtype": dtype, "p": p, "residual": residual}


def _ffn(direction, T, d, f, save, addend):
    return {"op": "ffn", "dir": direction, "T": T, "d": d, "f": f, "dtype": "bf16", "save": save, "addend": addend}


def listed():
    return [
        # the norm before the coarse workload's layer (T = 4 x 4096 tokens)
        {"name": "ln fwd coarse", **_ln("fwd", 16384, 2048, "bf16", "bf16")},
        # one new token of the high-sparsity model's width: latency
        {"name": "ln fwd one token", **_ln("fwd", 1, 7168, "f32", "f32")},
        # the fine-grained workload's norm, the residual's gradient joined in the same pass
        {"name": "ln bwd fine", **_ln("bwd", 32768, 1536, "bf16", "f32", True)},
        # a ragged batch of rows whose width no vector divides
        {"name": "ln bwd odd", **_ln("bwd", 1001, 1037, "f32", "f32")},
        # the residual dropout after the coarse workload's layer
        {"name": "dropout fwd coarse", **_dropout("fwd", 16384, 2048, "bf16", 0.1, True)},
        # its backward pass on an odd fp32 batch
        {"name": "dropout bwd odd", **_dropout("bwd", 999, 1001, "f32", 0.25, False)},
        # the shared expert on one new token: the weights' bytes and the latency
        {"name": "ffn fwd one token", **_ffn("fwd", 1, 2048, 1024, False, True)},
        # a decode batch at the high-sparsity model's widths
        {"name": "ffn fwd decode batch", **_ffn("fwd", 96, 7168, 2048, False, True)},
        # training: the shared expert of the coarse workload, H kept for the backward pass
        {"name": "ffn fwd coarse", **_ffn("fwd", 16384, 2048, 1024, True, True)},
        # training: the fine-grained workload's narrow expert on every token
        {"name": "ffn bwd fine", **_ffn("bwd", 32768, 1536, 256, True, True)},
        # a short ragged batch at widths that no tile divides
        {"name": "ffn bwd ragged", **_ffn("bwd", 1500, 1000, 680, True, False)},
        # training at the high-sparsity model's widths: the largest
        {"name": "ffn bwd sparse", **_ffn("bwd", 8192, 7168, 2048, True, False)},
    ]


def _log(rng, low, high):
    return int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))


def draw(rng):
    op, direction = rng.choice(("layernorm", "dropout", "ffn")), rng.choice(("fwd", "bwd"))
    dtype, flag = rng.choice(("f32", "bf16")), rng.random() < 0.5
    T = _log(rng, 1, 32768)
    if op == "ffn":
        d, f = 8 * _log(rng, 16, 896), 8 * _log(rng, 8, 256)
        return _ffn(direction, min(T, 8192 * 7168 * 2048 // (d * f)), d, f, direction == "bwd" or rng.random() < 0.5, flag)
    d = _log(rng, 16, 8192)
    T = min(T, 32768 * 2048 // d)
    if op == "layernorm":
        return _ln(direction, T, d, dtype, rng.choice(("f32", dtype)), flag and direction == "bwd")
    return _dropout(direction, T, d, dtype, round(rng.uniform(0.01, 0.6), 3), flag and direction == "fwd")


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(1_000_003 * seed + 17)
    dt, T, d = _TYPES[case["dtype"]], case["T"], case["d"]

    def normal(*shape, std=1.0, mean=0.0, dtype=dt):
        return (torch.randn(*shape, generator=gen, device="cuda") * std + mean).to(dtype)

    s = dict(case)
    if case["op"] == "layernorm":
        wt = _TYPES[case["wtype"]]
        # a residual stream: rows of different scale around a small offset
        s["x"] = (normal(T, d, dtype=torch.float32) * (0.5 + 2 * torch.rand(T, 1, generator=gen, device="cuda")) + 0.25).to(dt)
        s["w"], s["b"] = normal(d, std=0.1, mean=1.0, dtype=wt), normal(d, std=0.1, dtype=wt)
        if case["dir"] == "bwd":
            s["dy"] = normal(T, d)
            s["add"] = normal(T, d) if case["addend"] else None
            x = s["x"].double()
            mean = x.mean(1)
            s["mean"], s["rstd"] = mean.float(), ((x - mean[:, None]).square().mean(1) + _EPS).rsqrt().float()
    elif case["op"] == "dropout":
        s["x"] = normal(T, d)
        s["res"] = normal(T, d, std=2.0) if case["residual"] else None
        s["rng"] = torch.tensor([0x1234_5678_9ABC + seed, 3 * seed + 1], dtype=torch.int64, device="cuda")  # seed, offset (the step)
    else:
        f = case["f"]
        s["x"] = normal(T, d)
        s["w1"], s["w3"], s["w2"] = normal(d, f, std=0.02), normal(d, f, std=0.02), normal(f, d, std=0.02)
        s["add"] = normal(T, d) if case["addend"] else None
        if case["dir"] == "bwd":
            s["dout"] = normal(T, d)
            s["H"] = torch.cat([s["x"] @ s["w1"], s["x"] @ s["w3"]], 1)
    return s


def _plain_layernorm(s):
    x, w, b = s["x"].float(), s["w"].float(), s["b"].float()
    if s["dir"] == "fwd":
        mean = x.sum(1, keepdim=True) / s["d"]
        c = x - mean
        rstd = 1 / torch.sqrt((c * c).sum(1, keepdim=True) / s["d"] + _EPS)
        return {"y": (c * rstd * w + b).to(s["x"].dtype), "mean": mean[:, 0], "rstd": rstd[:, 0]}
    dy, rstd = s["dy"].float(), s["rstd"][:, None]
    xh = (x - s["mean"][:, None]) * rstd
    g = dy * w
    dx = rstd * (g - g.sum(1, keepdim=True) / s["d"] - xh * ((g * xh).sum(1, keepdim=True) / s["d"]))
    if s["add"] is not None:
        dx = dx + s["add"].float()
    return {"dx": dx.to(s["x"].dtype), "dweight": (dy * xh).sum(0), "dbias": dy.sum(0)}


def _plain_keep(rng, n, thr):
    """Which of n elements the counter-based generator keeps (32-bit words held in int64)."""
    low = 0xFFFFFFFF
    block = torch.arange((n + 7) // 8, device=rng.device)
    c0, c1, c2, c3 = block & low, block >> 32, rng[1] & low, (rng[1] >> 32) & low
    k0, k1 = rng[0] & low, (rng[0] >> 32) & low
    for _ in range(10):
        a, b = c0 * 0xD2511F53, c2 * 0xCD9E8D57  # the low 64 bits of the products: wrapped
        c0, c1, c2, c3 = ((b >> 32) & low) ^ c1 ^ k0, b & low, ((a >> 32) & low) ^ c3 ^ k1, a & low
        k0, k1 = (k0 + 0x9E3779B9) & low, (k1 + 0xBB67AE85) & low
    halves = [h for c in (c0, c1, c2, c3) for h in (c & 0xFFFF, c >> 16)]
    return torch.stack(halves, 1).reshape(-1)[:n] >= thr


def _plain_dropout(s):
    thr = round(s["p"] * 65536)
    keep = _plain_keep(s["rng"], s["x"].numel(), thr).view(s["x"].shape)
    out = torch.where(keep, s["x"].float() * (65536 / (65536 - thr)), 0.0)
    if s["res"] is not None:
        out = out + s["res"].float()
    return {"out": out.to(s["x"].dtype)}


def _plain_ffn(s):
    x, w1, w3, w2 = s["x"].float(), s["w1"].float(), s["w3"].float(), s["w2"].float()
    dt, f = s["x"].dtype, s["f"]
    add = 0.0 if s["add"] is None else s["add"].float()
    if s["dir"] == "fwd":
        h1, h3 = x @ w1, x @ w3
        y = (h1 / (1 + torch.exp(-h1)) * h3) @ w2 + add
        return {"y": y.to(dt), "H": torch.cat([h1, h3], 1).to(dt)} if s["save"] else {"y": y.to(dt)}
    dout, h1, h3 = s["dout"].float(), s["H"][:, :f].float(), s["H"][:, f:].float()
    sig = 1 / (1 + torch.exp(-h1))
    da = dout @ w2.T
    dh1, dh3 = da * h3 * (sig * (1 + h1 * (1 - sig))), da * h1 * sig
    return {"dx": (dh1 @ w1.T + dh3 @ w3.T + add).to(dt), "dw1": (x.T @ dh1).to(dt), "dw3": (x.T @ dh3).to(dt),
            "dw2": ((h1 * sig * h3).T @ dout).to(dt)}


def run(state):
    s = state
    if not own:
        return {"layernorm": _plain_layernorm, "dropout": _plain_dropout, "ffn": _plain_ffn}[s["op"]](s)
    from mixture_experts_layer_59_b200 import binding as B
    if s["op"] == "layernorm":
        if s["dir"] == "fwd":
            y, mean, rstd = B.moe_layernorm_fwd(s["x"], s["w"], s["b"], eps=_EPS)
            return {"y": y, "mean": mean, "rstd": rstd}
        g = B.moe_layernorm_bwd(s["dy"], s["x"], s["w"], s["mean"], s["rstd"], addend=s["add"])
        return {"dx": g["dx"], "dweight": g["dweight"], "dbias": g["dbias"]}
    if s["op"] == "dropout":
        if s["dir"] == "fwd":
            return {"out": B.moe_dropout_fwd(s["x"], s["p"], s["rng"], residual=s["res"])}
        return {"out": B.moe_dropout_bwd(s["x"], s["p"], s["rng"])}
    if s["dir"] == "fwd":
        y, H = B.moe_shared_ffn_fwd(s["x"], s["w1"], s["w3"], s["w2"], addend=s["add"], save=s["save"])
        return {"y": y, "H": H} if s["save"] else {"y": y}
    g = B.moe_shared_ffn_bwd(s["dout"], s["x"], s["w1"], s["w3"], s["w2"], s["H"], addend=s["add"])
    return {"dx": g["dx"], "dw1": g["dw1"], "dw3": g["dw3"], "dw2": g["dw2"]}


def work(case):
    T, d, e, fwd = case["T"], case["d"], _SIZE[case["dtype"]], case["dir"] == "fwd"
    n = T * d
    if case["op"] == "layernorm":
        we = _SIZE[case["wtype"]]
        if fwd:  # x; w, b; y, mean, rstd
            return {"bytes": 2 * n * e + 2 * d * we + 8 * T, "flops": 7 * n}
        # dy, x, addend, w, mean, rstd; dx, dweight, dbias
        return {"bytes": (4 if case["addend"] else 3) * n * e + d * we + 8 * T + 8 * d, "flops": 14 * n}
    if case["op"] == "dropout":
        return {"bytes": (3 if case["residual"] else 2) * n * e + 16, "flops": 2 * n}
    f, add = case["f"], 2 * n if case["addend"] else 0
    if fwd:  # x, W1, W3, W2, addend; y, H
        return {"bytes": 4 * n + 6 * d * f + add + (4 * T * f if case["save"] else 0), "flops": 6 * n * f}
    # dout, x, H, the weights, addend; dx, the weights' gradients
    return {"bytes": 6 * n + 4 * T * f + 12 * d * f + add, "flops": 12 * n * f}


def _exact_keep(seed, offset, n, thr):
    """The generator by its published rounds, in numpy's unsigned 64-bit integers, word by word."""
    u = np.uint64
    low, half = u(0xFFFFFFFF), u(32)
    index = np.arange(-(-n // 8), dtype=u)
    ctr = [index & low, index >> half, np.full_like(index, offset & 0xFFFFFFFF), np.full_like(index, offset >> 32)]
    key = [seed & 0xFFFFFFFF, seed >> 32]
    for _ in range(10):
        left, right = ctr[0] * u(0xD2511F53), ctr[2] * u(0xCD9E8D57)
        ctr = [(right >> half) ^ ctr[1] ^ u(key[0]), right & low, (left >> half) ^ ctr[3] ^ u(key[1]), left & low]
        key = [(key[0] + 0x9E3779B9) % 2**32, (key[1] + 0xBB67AE85) % 2**32]
    words = np.stack(ctr, axis=1).astype("<u4")
    return words.view("<u2").reshape(-1)[:n] >= thr


def exact(case, seed):
    s = prepare(case, seed)
    v = {k: t.double() for k, t in s.items() if isinstance(t, torch.Tensor) and t.is_floating_point()}
    if case["op"] == "layernorm":
        x = v["x"]
        if case["dir"] == "fwd":
            var, mean = torch.var_mean(x, dim=1, correction=0)
            rstd = (var + _EPS) ** -0.5
            return {"y": torch.addcmul(v["b"], (x - mean.unsqueeze(1)) * rstd.unsqueeze(1), v["w"]), "mean": mean, "rstd": rstd}
        mean, rstd, dy = v["mean"].unsqueeze(1), v["rstd"].unsqueeze(1), v["dy"]
        hat = (x - mean) * rstd
        g = dy * v["w"]
        dx = (g - g.mean(1, True) - hat * (g * hat).mean(1, True)) * rstd
        return {"dx": dx + v["add"] if "add" in v else dx, "dweight": torch.einsum("td,td->d", dy, hat), "dbias": dy.sum(0)}
    if case["op"] == "dropout":
        thr = round(case["p"] * 65536)
        seed_, offset = (int(i) for i in s["rng"].tolist())
        keep = torch.from_numpy(_exact_keep(seed_, offset, s["x"].numel(), thr)).to("cuda").view(s["x"].shape)
        out = torch.zeros_like(v["x"])
        out[keep] = v["x"][keep] / (1 - thr / 65536)
        return {"out": out + v["res"] if "res" in v else out}
    x, w1, w3, w2, add = v["x"], v["w1"], v["w3"], v["w2"], v.get("add", 0.0)
    if case["dir"] == "fwd":
        h1, h3 = x.mm(w1), x.mm(w3)
        y = torch.mm(h1 * torch.sigmoid(h1) * h3, w2) + add
        return {"y": y, "H": torch.cat((h1, h3), dim=1)} if case["save"] else {"y": y}
    h1, h3 = v["H"].split(case["f"], dim=1)
    gate = torch.sigmoid(h1)
    da = v["dout"].mm(w2.t())
    dh1, dh3 = da * h3 * (gate + h1 * gate * (1 - gate)), da * (h1 * gate)
    return {"dx": dh1.mm(w1.t()) + dh3.mm(w3.t()) + add, "dw1": x.t().mm(dh1), "dw3": x.t().mm(dh3),
            "dw2": (h1 * gate * h3).t().mm(v["dout"])}
