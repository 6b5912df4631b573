"""The dense operators beside the expert layer, case by case: their inputs, their plain
forms in elementary torch operations and the calls a program makes of this package.

Operators
  linear   out = act(x W^T + b) + residual, with the pre-activation kept for training
  linear_grad   its gradients: dx, dW, db from dL/dout
  ffn      the gated feed-forward block: out = (act(x Wg^T) * (x Wu^T)) W2^T + residual
  ffn_grad      its gradients: dx, dW13, dW2 from dL/dout
  clip     the global L2 norm over many gradient tensors, and the tensors scaled to it

x is [T, K] (rows may lie apart by more than K), weights are row-major [out, in];
w13 holds Wg's rows, then Wu's.
"""
import math

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
ACTS = ("none", "silu", "gelu", "gelu_tanh", "relu", "relu2")


# ----------------------------------------------------------------- cases ---

def listed():
    return [
        # one new token through an output projection of the decode width, added to the residual stream
        dict(name="linear_decode", op="linear", T=1, K=2048, N=2048, act="none", bias=False, residual=True, train=False,
             dtype="bf16", pad=0),
        # a prefill batch through a wide down projection with the residual
        dict(name="linear_prefill", op="linear", T=16384, K=8192, N=2048, act="none", bias=False, residual=True,
             train=False, dtype="bf16", pad=0),
        # an odd batch of a small model in fp16: bias, squared ReLU, rows apart, pre-activation kept for training
        dict(name="linear_ragged", op="linear", T=777, K=1000, N=1848, act="relu2", bias=True, residual=True, train=True,
             dtype="fp16", pad=24),
        # the training step of an ungated feed-forward's first projection
        dict(name="linear_grad_train", op="linear_grad", T=8192, K=2048, N=8192, act="gelu_tanh", bias=True,
             dtype="bf16", pad=0),
        # a short odd batch of a plain projection with bias, fp16
        dict(name="linear_grad_ragged", op="linear_grad", T=413, K=1352, N=680, act="none", bias=True, dtype="fp16",
             pad=8),
        # a verifier batch of three tokens: every weight is read once for three rows
        dict(name="ffn_decode", op="ffn", T=3, d=2048, F=6144, act="silu", residual=True, train=False, dtype="bf16",
             pad=0),
        # a batch of requests decoded together, on the width of the squared-ReLU layer, odd in every tile
        dict(name="ffn_batch", op="ffn", T=261, d=2688, F=1856, act="gelu", residual=False, train=True, dtype="bf16",
             pad=0),
        # prompt processing of a dense layer: the tensor cores' case
        dict(name="ffn_prefill", op="ffn", T=4096, d=4096, F=12288, act="silu", residual=True, train=False,
             dtype="bf16", pad=0),
        # a dense layer's training step
        dict(name="ffn_grad_train", op="ffn_grad", T=8192, d=2048, F=6144, act="silu", dtype="bf16", pad=0),
        # a short odd training batch
        dict(name="ffn_grad_ragged", op="ffn_grad", T=333, d=1016, F=1720, act="gelu_tanh", dtype="fp16", pad=16),
        # the gradients of a tiny layer: a dozen small tensors of three types, at any alignment
        dict(name="clip_small", op="clip", tensors=12, total=300_000, spread=2.0, types="mixed", max_norm=0.1),
        # the gradients of one expert layer of 128 experts of width 768 with its router and norms
        dict(name="clip_layer", op="clip", tensors=300, total=604_000_000, spread=3.0, types="bf16", max_norm=1.0),
    ]


MOST_FLOPS = 1.2e12
MOST_ELEMENTS = 604_000_000


def _log(rng, lo, hi, step=1):
    v = math.exp(rng.uniform(math.log(lo), math.log(hi + 1)))
    return max(lo, min(hi, int(v) // step * step or step))


def draw(rng):
    op = rng.choice(["linear", "linear", "linear_grad", "ffn", "ffn", "ffn_grad", "clip"])
    dtype = rng.choice(["bf16", "bf16", "fp16"])
    pad = rng.choice([0, 0, 8, 40])
    while op != "clip":
        T = _log(rng, 1, 16384)
        if op in ("linear", "linear_grad"):
            c = dict(op=op, T=T, K=_log(rng, 64, 8192, 8), N=_log(rng, 64, 16384, 8), act=rng.choice(ACTS),
                     bias=rng.random() < 0.5, dtype=dtype, pad=pad)
            if op == "linear":
                c.update(residual=rng.random() < 0.5, train=rng.random() < 0.5)
        else:
            c = dict(op=op, T=T, d=_log(rng, 64, 8192, 8), F=_log(rng, 64, 16384, 8), act=rng.choice(ACTS[1:5]),
                     dtype=dtype, pad=pad)
            if op == "ffn":
                c.update(residual=rng.random() < 0.5, train=rng.random() < 0.5)
        if work(c)["flops"] <= MOST_FLOPS:
            return c
    return dict(op="clip", tensors=_log(rng, 1, 3000), total=_log(rng, 4000, MOST_ELEMENTS // 4),
                spread=rng.uniform(0.0, 4.0), types=rng.choice(["bf16", "fp16", "fp32", "mixed"]),
                max_norm=rng.choice([0.1, 1.0, 1e6]))


# ------------------------------------------------------------------ work ---

def _sizes(case):
    """Element counts of the clipped tensors: `tensors` of them, log-spread, `total` together."""
    n, total = case["tensors"], case["total"]
    share = [math.exp(case["spread"] * math.sin(1.0 + 2.4 * i)) for i in range(n)]
    s = sum(share)
    sizes = [max(1, int(total * v / s)) for v in share]
    if case["types"] == "mixed":
        return [(v, ("bf16", "fp32", "fp16")[i % 3]) for i, v in enumerate(sizes)]
    return [(v, case["types"]) for v in sizes]


def work(case):
    op = case["op"]
    if op == "clip":
        b = sum(v * (4 if t == "fp32" else 2) for v, t in _sizes(case))
        return {"bytes": 2 * b + 4, "flops": 3 * sum(v for v, _ in _sizes(case))}
    T = case["T"]
    if op in ("linear", "linear_grad"):
        K, N = case["K"], case["N"]
        if op == "linear":
            e = T * K + N * K + T * N * (1 + case["residual"] + case["train"]) + N * case["bias"]
            return {"bytes": 2 * e, "flops": 2 * T * N * K}
        e = 2 * (T * K + N * K) + T * N * (1 + (case["act"] != "none")) + N * case["bias"]
        return {"bytes": 2 * e, "flops": 4 * T * N * K}
    d, F = case["d"], case["F"]
    if op == "ffn":
        e = T * d * (2 + case["residual"]) + 3 * d * F + T * 2 * F * case["train"]
        return {"bytes": 2 * e, "flops": 6 * T * d * F}
    return {"bytes": 2 * (3 * T * d + 6 * d * F + 2 * T * F), "flops": 12 * T * d * F}


# --------------------------------------------------------------- prepare ---

def _inputs(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)

    def normal(shape, std, dtype):
        return (torch.randn(shape, generator=gen, device="cuda", dtype=torch.float32) * std).to(dtype)

    if case["op"] == "clip":
        pairs = _sizes(case)
        flat = {}
        for t in sorted({t for _, t in pairs}):
            flat[t] = normal((sum(v for v, u in pairs if u == t),), 1e-3, DTYPES[t])
        at = dict.fromkeys(flat, 0)
        grads = []
        for i, (v, t) in enumerate(pairs):
            g = flat[t][at[t]:at[t] + v]
            g.mul_(2.0 ** (i % 5 - 2))  # layers' gradients differ in size
            grads.append(g)
            at[t] += v
        return dict(grads=grads, flat=flat, types=[t for _, t in pairs])

    dt = DTYPES[case["dtype"]]
    T, pad = case["T"], case["pad"]

    def rows(n, std=1.0):
        return normal((T, n + pad), std, dt)[:, :n]

    if case["op"] in ("linear", "linear_grad"):
        K, N = case["K"], case["N"]
        s = dict(x=rows(K), w=normal((N, K), 0.02, dt), bias=normal((N,), 0.1, dt) if case["bias"] else None)
        if case["op"] == "linear":
            s["residual"] = rows(N) if case["residual"] else None
        else:
            # the pre-activations the forward kept: of the size that 0.02-weights give
            s["pre"] = normal((T, N), 0.02 * math.sqrt(K), dt) if case["act"] != "none" else None
            s["dout"] = rows(N)
        return s
    d, F = case["d"], case["F"]
    s = dict(x=rows(d), w13=normal((2 * F, d), 0.02, dt), w2=normal((d, F), 0.02, dt))
    if case["op"] == "ffn":
        s["residual"] = rows(d) if case["residual"] else None
    else:
        s["pre"] = normal((T, 2 * F), 0.02 * math.sqrt(d), dt)
        s["dout"] = rows(d)
    return s


def prepare(case, seed):
    s = _inputs(case, seed)
    s["case"] = case
    if own:  # the buffers and the plan that a program keeps
        from grouped_gemm_gating_b200 import moe as M
        if case["op"] == "clip":
            s["out"] = {t: torch.empty_like(v) for t, v in s["flat"].items()}
            at = dict.fromkeys(s["out"], 0)
            outs = []
            for g, t in zip(s["grads"], s["types"]):
                outs.append(s["out"][t][at[t]:at[t] + g.numel()])
                at[t] += g.numel()
            s["plan"] = M.GradClip(s["grads"], outs)
        else:
            act = getattr(M, "EPI_" + case["act"].upper())
            dt, T = DTYPES[case["dtype"]], case["T"]
            train = case["op"].endswith("_grad") or case["train"]
            if "K" in case:
                s["buf"] = M.LinearBuffers(T, case["K"], case["N"], act, dtype=dt, train=train, bias=case["bias"])
            else:
                s["buf"] = M.FFNBuffers(T, case["d"], case["F"], act, dtype=dt, train=train)
    return s


# ----------------------------------------------------------- plain forms ---

def _act(z, name):
    if name == "none":
        return z
    if name == "silu":
        return z / (1 + torch.exp(-z))
    if name == "gelu":
        return 0.5 * z * (1 + torch.erf(z * math.sqrt(0.5)))
    if name == "gelu_tanh":
        return 0.5 * z * (1 + torch.tanh(math.sqrt(2 / math.pi) * (z + 0.044715 * z * z * z)))
    p = z * (z > 0)
    return p if name == "relu" else p * p


def _act_slope(z, name):
    if name == "none":
        return torch.ones_like(z)
    if name == "silu":
        s = 1 / (1 + torch.exp(-z))
        return s * (1 + z * (1 - s))
    if name == "gelu":
        return 0.5 * (1 + torch.erf(z * math.sqrt(0.5))) + z * torch.exp(-0.5 * z * z) / math.sqrt(2 * math.pi)
    if name == "gelu_tanh":
        c = math.sqrt(2 / math.pi)
        t = torch.tanh(c * (z + 0.044715 * z * z * z))
        return 0.5 * (1 + t) + 0.5 * z * (1 - t * t) * c * (1 + 3 * 0.044715 * z * z)
    return (z > 0).float() if name == "relu" else 2 * z * (z > 0)


def _plain_linear(s, c):
    z = s["x"].float() @ s["w"].float().T
    if s["bias"] is not None:
        z = z + s["bias"].float()
    y = _act(z, c["act"])
    if s["residual"] is not None:
        y = y + s["residual"].float()
    dt = s["x"].dtype
    out = {"out": y.to(dt)}
    if c["train"] and c["act"] != "none":
        out["pre"] = z.to(dt)
    return out


def _plain_linear_grad(s, c):
    dt = s["x"].dtype
    dz = s["dout"].float()
    if c["act"] != "none":
        dz = dz * _act_slope(s["pre"].float(), c["act"])
    out = {"dx": (dz @ s["w"].float()).to(dt), "dw": (dz.T @ s["x"].float()).to(dt)}
    if c["bias"]:
        out["dbias"] = dz.sum(0).to(dt)
    return out


def _plain_ffn(s, c):
    dt, F = s["x"].dtype, c["F"]
    z = s["x"].float() @ s["w13"].float().T
    y = (_act(z[:, :F], c["act"]) * z[:, F:]) @ s["w2"].float().T
    if s["residual"] is not None:
        y = y + s["residual"].float()
    out = {"out": y.to(dt)}
    if c["train"]:
        out["pre"] = z.to(dt)
    return out


def _plain_ffn_grad(s, c):
    dt, F = s["x"].dtype, c["F"]
    g, u = s["pre"][:, :F].float(), s["pre"][:, F:].float()
    dy = s["dout"].float()
    a = _act(g, c["act"])
    dh = dy @ s["w2"].float()
    dz = torch.cat([dh * u * _act_slope(g, c["act"]), dh * a], 1)
    return {"dx": (dz @ s["w13"].float()).to(dt), "dw13": (dz.T @ s["x"].float()).to(dt),
            "dw2": (dy.T @ (a * u)).to(dt)}


def _plain_clip(s, c):
    norm = torch.stack([g.float().square().sum(dtype=torch.float64) for g in s["grads"]]).sum().sqrt()
    scale = torch.clamp(c["max_norm"] / (norm + 1e-6), max=1.0).float()
    scaled = [(g.float() * scale).to(g.dtype) for g in s["grads"]]
    out = {t: torch.cat([v for v, u in zip(scaled, s["types"]) if u == t]) for t in s["flat"]}
    return {"norm": norm.float(), "grads": out}


# ------------------------------------------------------------------- run ---

def run(state):
    c, s = state["case"], state
    op = c["op"]
    if not own:
        return {"linear": _plain_linear, "linear_grad": _plain_linear_grad, "ffn": _plain_ffn,
                "ffn_grad": _plain_ffn_grad, "clip": _plain_clip}[op](s, c)
    if op == "clip":
        norm = s["plan"].clip(c["max_norm"])
        return {"norm": norm, "grads": s["out"]}
    b = s["buf"]
    if op == "linear":
        out = {"out": b.forward(s["x"], s["w"], s["bias"], s["residual"])}
        if c["train"] and c["act"] != "none":
            out["pre"] = b.pre
        return out
    if op == "linear_grad":
        b.backward(s["x"], s["w"], s["dout"], pre=s["pre"])
        out = {"dx": b.dx, "dw": b.dw}
        if c["bias"]:
            out["dbias"] = b.dbias
        return out
    if op == "ffn":
        out = {"out": b.forward(s["x"], s["w13"], s["w2"], s["residual"])}
        if c["train"]:
            out["pre"] = b.pre
        return out
    b.backward(s["x"], s["w13"], s["w2"], s["dout"], pre=s["pre"])
    return {"dx": b.dx, "dw13": b.dw13, "dw2": b.dw2}


# ----------------------------------------------------------------- exact ---

def _value_and_slope(z, name):
    """(act(z), act'(z)) in 64 bits, from the activations' definitions."""
    one = torch.ones_like(z)
    if name == "none":
        return z, one
    if name == "silu":
        sig = torch.special.expit(z)
        return z * sig, sig + z * sig * torch.special.expit(-z)
    if name == "gelu":
        phi = torch.special.ndtr(z)
        return z * phi, phi + z * torch.exp(-z * z / 2) * (2 * math.pi) ** -0.5
    if name == "gelu_tanh":
        # (1 + tanh v) / 2 is the logistic function of 2 v
        k = 2 * (2 / math.pi) ** 0.5
        sig = torch.special.expit(k * (z + 0.044715 * z ** 3))
        return z * sig, sig + z * sig * (1 - sig) * k * (1 + 0.134145 * z ** 2)
    p = torch.clamp(z, min=0)
    return (p, (z > 0).double()) if name == "relu" else (p * p, 2 * p)


def exact(case, seed):
    s = {k: v.double() if isinstance(v, torch.Tensor) else v for k, v in _inputs(case, seed).items()}
    op = case["op"]
    if op == "clip":
        flat = {t: v.double() for t, v in s["flat"].items()}
        norm = math.sqrt(sum(float(torch.dot(v, v)) for v in flat.values()))
        scale = min(1.0, case["max_norm"] / (norm + 1e-6))
        return {"norm": torch.tensor(norm, dtype=torch.float64), "grads": {t: v * scale for t, v in flat.items()}}
    if op == "linear":
        z = torch.einsum("tk,nk->tn", s["x"], s["w"])
        if s["bias"] is not None:
            z += s["bias"]
        y = _value_and_slope(z, case["act"])[0]
        out = {"out": y if s["residual"] is None else s["residual"] + y}
        if case["train"] and case["act"] != "none":
            out["pre"] = z
        return out
    if op == "linear_grad":
        e = s["dout"] if s["pre"] is None else s["dout"] * _value_and_slope(s["pre"], case["act"])[1]
        out = {"dx": torch.einsum("tn,nk->tk", e, s["w"]), "dw": torch.einsum("tn,tk->nk", e, s["x"])}
        if case["bias"]:
            out["dbias"] = torch.einsum("tn->n", e)
        return out
    F = case["F"]
    wg, wu = s["w13"][:F], s["w13"][F:]
    if op == "ffn":
        g, u = torch.einsum("td,fd->tf", s["x"], wg), torch.einsum("td,fd->tf", s["x"], wu)
        y = torch.einsum("tf,df->td", _value_and_slope(g, case["act"])[0] * u, s["w2"])
        out = {"out": y if s["residual"] is None else s["residual"] + y}
        if case["train"]:
            out["pre"] = torch.cat([g, u], dim=1)
        return out
    g, u = s["pre"].split(F, dim=1)
    a, slope = _value_and_slope(g, case["act"])
    dh = torch.einsum("td,df->tf", s["dout"], s["w2"])
    eg, eu = dh * u * slope, dh * a
    return {"dx": torch.einsum("tf,fd->td", eg, wg) + torch.einsum("tf,fd->td", eu, wu),
            "dw13": torch.cat([torch.einsum("tf,td->fd", eg, s["x"]), torch.einsum("tf,td->fd", eu, s["x"])]),
            "dw2": torch.einsum("td,tf->df", s["dout"], a * u)}
