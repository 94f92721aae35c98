"""Timed cases of the dense sub-block operators: layer norm, linear layer, dropout.

These are the pieces of a pre-norm feed-forward sub-block of the OPT kind on retained rows
(layer norm -> product with bias and ReLU -> product with bias -> dropout -> residual) and
their gradients.  With ``own`` false, ``run`` computes each operator from elementary torch
operations in 32 bits, rounded once at the end; with ``own`` true it makes the library calls.
``exact`` restates the definitions in 64 bits.

Shapes: hidden 256 / 4096 / 5120 and feed-forward width 11008, segments of 4096 rows,
26240 retained rows of a 32768-token sequence in blocks of 128.
"""
import math

import numpy as np
import torch

own = False


def _lib():
    import token_sparse_long_b200
    return token_sparse_long_b200


_DT = {"f32": torch.float32, "bf16": torch.bfloat16}
_BYTES = {"f32": 4, "bf16": 2}
_EPS = 1e-5


# ------------------------------------------------------------------ cases
def listed():
    return [
        # the small fp32 workload's activations (512 tokens, hidden 256): latency counts
        dict(name="ln_fwd_512x256_f32", op="ln_fwd", rows=512, h=256, dt="f32", wdt="f32", blk=0, S=0),
        # retained rows of a 32K-token sequence read through the block list, hidden 4096
        dict(name="ln_fwd_kept_26240x4096", op="ln_fwd", rows=26240, h=4096, dt="bf16", wdt="bf16", blk=128, S=32768),
        # odd width and row count in fp32: no row but the first is 16-byte aligned
        dict(name="ln_bwd_777x1001_f32", op="ln_bwd", rows=777, h=1001, dt="f32", wdt="f32", res=False),
        # one backward segment of 4096 rows
        dict(name="ln_bwd_4096x4096", op="ln_bwd", rows=4096, h=4096, dt="bf16", wdt="bf16", res=False),
        # every retained row at the 13B width, residual gradient added in the same pass
        dict(name="ln_bwd_26240x5120_res", op="ln_bwd", rows=26240, h=5120, dt="bf16", wdt="bf16", res=True),
        # one token through the widening product (weights are all the traffic)
        dict(name="lin_fwd_1_up_relu", op="lin_fwd", M=1, K=4096, N=11008, act="relu", bdt="bf16", res=False, pre=False),
        # a training segment through the widening product, pre-activation saved for the backward
        dict(name="lin_fwd_4096_up_gelu", op="lin_fwd", M=4096, K=4096, N=11008, act="gelu", bdt="bf16", res=False,
             pre=True),
        # all retained rows through the narrowing product with the residual add
        dict(name="lin_fwd_26240_down_res", op="lin_fwd", M=26240, K=11008, N=4096, act="none", bdt="bf16", res=True,
             pre=False),
        # ragged sizes, smooth activation: input, weight and bias gradients
        dict(name="lin_bwd_1000x520x1541_gelu", op="lin_bwd", M=1000, K=520, N=1541, act="gelu"),
        # a training segment's gradients through the widening product
        dict(name="lin_bwd_4096_up_relu", op="lin_bwd", M=4096, K=4096, N=11008, act="relu"),
        # small fp32 dropout: latency counts
        dict(name="dropout_512x256_f32", op="dropout", rows=512, h=256, dt="f32", p=0.1, res=False, blk=0, S=0),
        # every retained row with the residual add, mask keyed by the sequence position
        dict(name="dropout_26240x4096_res", op="dropout", rows=26240, h=4096, dt="bf16", p=0.1, res=True, blk=128,
             S=32768),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["ln_fwd", "ln_bwd", "lin_fwd", "lin_bwd", "dropout"])
    if op in ("lin_fwd", "lin_bwd"):
        K = max(64, _log(rng, 64, 11008) // 8 * 8)  # rows of x and w start 16-byte aligned
        N = _log(rng, 64, 11008)
        if rng.random() < 0.6:
            N = max(64, N // 64 * 64)
        top = 26240 * 4096 * 11008 // (2 if op == "lin_bwd" else 1)
        M = _log(rng, 1, max(1, min(26240, top // (K * N))))
        c = dict(op=op, M=M, K=K, N=N, act=rng.choice(["none", "relu", "gelu", "silu"]))
        if op == "lin_fwd":
            c.update(bdt=rng.choice(["f32", "bf16"]), res=rng.random() < 0.5, pre=rng.random() < 0.3)
        return c
    h = _log(rng, 64, 8192)
    if rng.random() < 0.6:
        h = max(64, h // 64 * 64)
    dt = rng.choice(["f32", "bf16"])
    blk, S = 0, 0
    rows = _log(rng, 1, 32768)
    if op != "ln_bwd" and rng.random() < 0.5:
        blk = rng.choice([32, 64, 128])
        n = max(1, rows // blk)
        rows, S = n * blk, (n + rng.randrange(0, n + 1)) * blk
    if op == "ln_fwd":
        return dict(op=op, rows=rows, h=h, dt=dt, wdt=rng.choice([dt, "f32"]), blk=blk, S=S)
    if op == "ln_bwd":
        return dict(op=op, rows=rows, h=h, dt=dt, wdt=rng.choice([dt, "f32"]), res=rng.random() < 0.5)
    return dict(op=op, rows=rows, h=h, dt=dt, p=round(rng.uniform(0.02, 0.6), 3), res=rng.random() < 0.5, blk=blk, S=S)


# ------------------------------------------------------------------ inputs
def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(int(seed))


def _randn(g, shape, dt=torch.float32, scale=1.0, shift=0.0):
    t = torch.randn(shape, generator=g, device="cuda", dtype=torch.float32)
    return t.mul_(scale).add_(shift).to(dt)


def _kept(g, case):
    """Ascending random block list, its device count, block length (none without a list)."""
    if not case["blk"]:
        return None, None, 1
    nb, n = case["S"] // case["blk"], case["rows"] // case["blk"]
    idx = torch.randperm(nb, generator=g, device="cuda")[:n].sort().values.to(torch.int32)
    return idx, torch.tensor([n], dtype=torch.int32, device="cuda"), case["blk"]


def prepare(case, seed):
    g = _gen(seed)
    op = case["op"]
    st = {"op": op, "case": case}
    if op in ("ln_fwd", "ln_bwd"):
        dt, wdt, h = _DT[case["dt"]], _DT[case["wdt"]], case["h"]
        rows = case["S"] if op == "ln_fwd" and case["blk"] else case["rows"]
        # residual-stream rows: scales differ from row to row, a few columns sit off centre
        x = _randn(g, (rows, h))
        x *= torch.exp(0.5 * torch.randn(rows, 1, generator=g, device="cuda"))
        x += _randn(g, (1, h), scale=0.5)
        st["x"] = x.to(dt)
        st["gamma"] = _randn(g, (h,), wdt, 0.1, 1.0)
        if op == "ln_fwd":
            st["beta"] = _randn(g, (h,), wdt, 0.1)
            st["idx"], st["n_kept"], st["blk"] = _kept(g, case)
        else:
            x64 = st["x"].double()
            mean = x64.mean(1, keepdim=True)
            st["mean"] = mean[:, 0].float()
            st["rstd"] = torch.rsqrt((x64 - mean).square_().mean(1) + _EPS).float()
            st["dy"] = _randn(g, (rows, h), dt)
            st["dres"] = _randn(g, (rows, h), dt) if case["res"] else None
    elif op in ("lin_fwd", "lin_bwd"):
        M, K, N = case["M"], case["K"], case["N"]
        bf = torch.bfloat16
        st["x"] = _randn(g, (M, K), bf)
        st["w"] = _randn(g, (N, K), bf, 1.3 / math.sqrt(K))
        st["act"] = case["act"]
        if op == "lin_fwd":
            st["bias"] = _randn(g, (N,), _DT[case["bdt"]], 0.1)
            st["res"] = _randn(g, (M, N), bf) if case["res"] else None
            st["pre"] = case["pre"]
        else:
            st["dy"] = _randn(g, (M, N), bf)
            st["z"] = None if case["act"] == "none" else (st["x"] @ st["w"].T + _randn(g, (N,), bf, 0.1))
    else:
        rows, h, dt = case["rows"], case["h"], _DT[case["dt"]]
        st["x"] = _randn(g, (rows, h), dt)
        st["res"] = _randn(g, (rows, h), dt) if case["res"] else None
        st["idx"], st["n_kept"], st["blk"] = _kept(g, case)
        st["p"] = case["p"]
        st["seed"] = int(seed) * 2654435761 + 12345
        st["offset"] = int(seed) + (7 << 33)
    return st


# ------------------------------------------------------------------ plain forms
def _positions(st, rows):
    """Sequence row of every compact row."""
    r = torch.arange(rows, device="cuda")
    if st["idx"] is None:
        return r
    return st["idx"].long()[r // st["blk"]] * st["blk"] + r % st["blk"]


def _ln_fwd(st):
    x = st["x"]
    if st["idx"] is not None:
        x = x[_positions(st, st["case"]["rows"])]
    x = x.float()
    mean = x.mean(1, keepdim=True)
    d = x - mean
    rstd = 1.0 / torch.sqrt((d * d).mean(1, keepdim=True) + _EPS)
    y = d * rstd * st["gamma"].float() + st["beta"].float()
    return {"y": y.to(st["x"].dtype), "mean": mean[:, 0], "rstd": rstd[:, 0]}


def _ln_bwd(st):
    dy = st["dy"].float()
    xhat = (st["x"].float() - st["mean"][:, None]) * st["rstd"][:, None]
    gy = dy * st["gamma"].float()
    dx = st["rstd"][:, None] * (gy - gy.mean(1, keepdim=True) - xhat * (gy * xhat).mean(1, keepdim=True))
    if st["dres"] is not None:
        dx = dx + st["dres"].float()
    return {"dx": dx.to(st["x"].dtype), "dgamma": (dy * xhat).sum(0), "dbeta": dy.sum(0)}


def _act(z, act):
    if act == "relu":
        return torch.where(z > 0, z, torch.zeros_like(z))
    if act == "gelu":
        return 0.5 * z * (1.0 + torch.erf(z * math.sqrt(0.5)))
    if act == "silu":
        return z / (1.0 + torch.exp(-z))
    return z


def _act_grad(z, act):
    if act == "relu":
        return (z > 0).float()
    if act == "gelu":
        return 0.5 * (1.0 + torch.erf(z * math.sqrt(0.5))) + z * torch.exp(-0.5 * z * z) / math.sqrt(2 * math.pi)
    s = 1.0 / (1.0 + torch.exp(-z))
    return s * (1.0 + z * (1.0 - s))


def _lin_fwd(st):
    z = st["x"].float() @ st["w"].float().T + st["bias"].float()
    y = _act(z, st["act"])
    if st["res"] is not None:
        y = y + st["res"].float()
    out = {"y": y.to(torch.bfloat16)}
    if st["pre"]:
        out["pre"] = z.to(torch.bfloat16)
    return out


def _lin_bwd(st):
    dz = st["dy"].float()
    if st["z"] is not None:
        dz = dz * _act_grad(st["z"].float(), st["act"])
    return {"dx": (dz @ st["w"].float()).to(torch.bfloat16), "dw": dz.T @ st["x"].float(), "db": dz.sum(0)}


def _mul_hi_lo(a, m):
    """High and low words of the 64-bit product of a 32-bit word (int64 tensor) and constant m."""
    p1, p2 = a * (m & 0xFFFF), a * (m >> 16)
    return (p2 + (p1 >> 16)) >> 16, ((p2 << 16) + p1) & 0xFFFFFFFF


def _keep_mask(pos, h, p, seed, offset):
    """Philox4x32-10 with counter (column group of 8, position, offset) and the seed as key:
    16 random bits an element, kept when they are at least round(p 2^16)."""
    c0 = torch.arange((h + 7) // 8, device="cuda")[None, :].expand(len(pos), -1)
    c1 = pos[:, None].expand_as(c0)
    c2 = torch.full_like(c0, offset & 0xFFFFFFFF)
    c3 = torch.full_like(c0, (offset >> 32) & 0xFFFFFFFF)
    k0, k1 = seed & 0xFFFFFFFF, (seed >> 32) & 0xFFFFFFFF
    for _ in range(10):
        h0, l0 = _mul_hi_lo(c0, 0xD2511F53)
        h1, l1 = _mul_hi_lo(c2, 0xCD9E8D57)
        c0, c1, c2, c3 = h1 ^ c1 ^ k0, l1, h0 ^ c3 ^ k1, l0
        k0, k1 = (k0 + 0x9E3779B9) & 0xFFFFFFFF, (k1 + 0xBB67AE85) & 0xFFFFFFFF
    bits = torch.stack([c0 & 0xFFFF, c0 >> 16, c1 & 0xFFFF, c1 >> 16, c2 & 0xFFFF, c2 >> 16, c3 & 0xFFFF, c3 >> 16], 2)
    return bits.reshape(len(pos), -1)[:, :h] >= math.floor(p * 65536 + 0.5)


def _dropout(st):
    x = st["x"]
    rows, h = x.shape
    keep = _keep_mask(_positions(st, rows), h, st["p"], st["seed"], st["offset"])
    scale = 65536.0 / (65536 - math.floor(st["p"] * 65536 + 0.5))
    y = torch.where(keep, x.float() * scale, torch.zeros((), device="cuda"))
    if st["res"] is not None:
        y = y + st["res"].float()
    return {"y": y.to(x.dtype)}


def run(state):
    st = state
    op = st["op"]
    if not own:
        return {"ln_fwd": _ln_fwd, "ln_bwd": _ln_bwd, "lin_fwd": _lin_fwd, "lin_bwd": _lin_bwd, "dropout": _dropout}[op](st)
    J = _lib()
    if op == "ln_fwd":
        n_max = None if st["idx"] is None else st["idx"].numel()
        y, mean, rstd = J.jenga_layernorm_fwd(st["x"], st["gamma"], st["beta"], eps=_EPS, idx=st["idx"],
                                              n_kept=st["n_kept"], blk=st["blk"], n_kept_max=n_max)
        return {"y": y, "mean": mean, "rstd": rstd}
    if op == "ln_bwd":
        dx, dg, db = J.jenga_layernorm_bwd(st["dy"], st["x"], st["mean"], st["rstd"], st["gamma"], dres=st["dres"])
        return {"dx": dx, "dgamma": dg, "dbeta": db}
    if op == "lin_fwd":
        y, pre = J.jenga_linear_fwd(st["x"], st["w"], st["bias"], act=st["act"], residual=st["res"], save_pre=st["pre"])
        return {"y": y, "pre": pre} if st["pre"] else {"y": y}
    if op == "lin_bwd":
        dx, dw, db = J.jenga_linear_bwd(st["dy"], st["x"], st["w"], act=st["act"], pre=st["z"])
        return {"dx": dx, "dw": dw, "db": db}
    return {"y": J.jenga_dropout(st["x"], st["p"], st["seed"], st["offset"], residual=st["res"], idx=st["idx"],
                                 n_kept=st["n_kept"], blk=st["blk"])}


# ------------------------------------------------------------------ work
def work(case):
    op = case["op"]
    if op in ("lin_fwd", "lin_bwd"):
        M, K, N = case["M"], case["K"], case["N"]
        if op == "lin_fwd":
            b = 2 * (M * K + N * K + M * N * (1 + case["res"] + case["pre"])) + _BYTES[case["bdt"]] * N
            return {"bytes": b, "flops": 2 * M * N * K}
        b = 2 * (M * N * (1 if case["act"] == "none" else 2) + 2 * M * K + N * K) + 4 * (N * K + N)
        return {"bytes": b, "flops": 4 * M * N * K}
    n, e = case["rows"] * case["h"], _BYTES[case["dt"]]
    if op == "ln_fwd":
        return {"bytes": 2 * n * e + 8 * case["rows"] + 2 * case["h"] * _BYTES[case["wdt"]], "flops": 8 * n}
    if op == "ln_bwd":
        return {"bytes": (3 + case["res"]) * n * e + 8 * case["rows"] + case["h"] * (_BYTES[case["wdt"]] + 8),
                "flops": 14 * n}
    return {"bytes": (2 + case["res"]) * n * e, "flops": 2 * n}


# ------------------------------------------------------------------ definitions in 64 bits
def _exact_philox(words, key):
    """Philox4x32-10 on numpy uint64 arrays holding 32-bit words."""
    m32, s32 = np.uint64(0xFFFFFFFF), np.uint64(32)
    a, b, c, d = words
    ka, kb = key
    for r in range(10):
        pa, pc = a * np.uint64(0xD2511F53), c * np.uint64(0xCD9E8D57)
        ra = np.uint64((ka + r * 0x9E3779B9) % (1 << 32))
        rb = np.uint64((kb + r * 0xBB67AE85) % (1 << 32))
        a, b, c, d = (pc >> s32) ^ b ^ ra, pc & m32, (pa >> s32) ^ d ^ rb, pa & m32
    return a, b, c, d


def exact(case, seed):
    st = prepare(case, seed)
    op = st["op"]
    f8 = torch.float64
    if op in ("ln_fwd", "ln_bwd"):
        x, gamma = st["x"].to(f8), st["gamma"].to(f8)
        if op == "ln_fwd":
            if st["idx"] is not None:
                x = x.view(-1, st["blk"], case["h"])[st["idx"].long()].reshape(case["rows"], case["h"])
            var, mean = torch.var_mean(x, 1, correction=0, keepdim=True)
            rstd = (var + _EPS).pow(-0.5)
            return {"y": torch.addcmul(st["beta"].to(f8), (x - mean) * rstd, gamma), "mean": mean[:, 0], "rstd": rstd[:, 0]}
        dy, rstd = st["dy"].to(f8), st["rstd"].to(f8)[:, None]
        n = (x - st["mean"].to(f8)[:, None]) * rstd
        c1 = (dy @ gamma)[:, None] / case["h"]
        c2 = ((dy * n) @ gamma)[:, None] / case["h"]
        dx = rstd * (dy * gamma - c1 - n * c2)
        if st["dres"] is not None:
            dx += st["dres"].to(f8)
        return {"dx": dx, "dgamma": torch.einsum("rh,rh->h", dy, n), "dbeta": dy.sum(0)}
    if op in ("lin_fwd", "lin_bwd"):
        x, w = st["x"].to(f8), st["w"].to(f8)
        if op == "lin_fwd":
            z = torch.addmm(st["bias"].to(f8), x, w.t())
            y = {"none": lambda t: t, "relu": lambda t: t.clamp(min=0), "silu": lambda t: t * torch.sigmoid(t),
                 "gelu": lambda t: t * torch.special.ndtr(t)}[case["act"]](z)
            out = {"y": y if st["res"] is None else y + st["res"].to(f8)}
            if st["pre"]:
                out["pre"] = z
            return out
        dz = st["dy"].to(f8)
        if case["act"] != "none":
            t = st["z"].to(f8)
            if case["act"] == "relu":
                dz = dz.masked_fill(t <= 0, 0.0)
            elif case["act"] == "gelu":
                dz = dz * (torch.special.ndtr(t) + t * torch.exp(-t.square() / 2) / math.sqrt(2 * math.pi))
            else:
                s = torch.sigmoid(t)
                dz = dz * (s + t * s * (1 - s))
        return {"dx": dz.mm(w), "dw": dz.t().mm(x), "db": dz.sum(0)}
    rows, h = case["rows"], case["h"]
    if case["blk"]:
        pos = (st["idx"].cpu().numpy().astype(np.uint64)[:, None] * np.uint64(case["blk"])
               + np.arange(case["blk"], dtype=np.uint64)[None, :]).reshape(-1)
    else:
        pos = np.arange(rows, dtype=np.uint64)
    q = (h + 7) // 8
    col, row = np.broadcast_arrays(np.arange(q, dtype=np.uint64)[None, :], pos[:, None])
    lo, hi = st["offset"] % (1 << 32), (st["offset"] >> 32) % (1 << 32)
    words = _exact_philox((col, row, np.full((1, 1), lo, np.uint64), np.full((1, 1), hi, np.uint64)),
                          (st["seed"] % (1 << 32), (st["seed"] >> 32) % (1 << 32)))
    t = int(math.floor(st["p"] * 65536 + 0.5))
    lanes = np.empty((rows, q, 8), dtype=bool)
    for i, v in enumerate(words):
        lanes[:, :, 2 * i] = (v & np.uint64(0xFFFF)) >= t
        lanes[:, :, 2 * i + 1] = (v >> np.uint64(16)) >= t
    keep = torch.from_numpy(lanes.reshape(rows, 8 * q)[:, :h]).to("cuda")
    y = st["x"].to(f8).masked_fill(~keep, 0.0) * (65536.0 / (65536 - t))
    return {"y": y if st["res"] is None else y + st["res"].to(f8)}
