"""Cases, inputs and plain forms of the 8-bit linear, the RMS norm and the
many-tensor AdamW step.

Four operators of the library, as a training or serving program calls them:

  fp8_fwd   y = x W^T through an e4m3 weight with one scale per 128 x 128
            block and rows in 8 bits with one scale per 128 columns
  fp8_bwd   dX = dY W through the same weight
  norm      RMS norm with the residual's addition; output bf16, or 8-bit rows
  norm_bwd  its gradients
  adamw     AdamW over many tensors, states in 32 bits or in 8

With `own` false, `run` computes the plain form: elementary torch operations
in fp32, rounded once at the end. With `own` true it makes the library calls.
`exact` evaluates the definitions in fp64.
"""

import math

import numpy as np
import torch

own = False

BLOCK = 128            # columns per scale of a row, rows and columns per scale of a weight
STATE_BLOCK = 256      # values per scale of an 8-bit optimizer state
TOP = {"e4m3": 448.0, "e5m2": 57344.0}
FP8 = {"e4m3": torch.float8_e4m3fn, "e5m2": torch.float8_e5m2}
LEAST = 2.0 ** -100    # smallest block maximum that a scale is made from

# the optimizer's hyperparameters are fp32 numbers
LR, BETA1, BETA2, EPS, DECAY = (float(np.float32(v)) for v in (1e-4, 0.9, 0.999, 1e-8, 0.01))
STEP = 120
NORM_EPS = float(np.float32(1e-5))


# ---------------------------------------------------------------- cases
def listed():
    return [
        # one generated token through a square projection
        {"name": "linear, one token", "op": "fp8_fwd", "m": 1, "n": 4096, "k": 4096, "fmt": "e4m3", "rows": "bf16"},
        # a batch of 37 sequences, one token each, through the wide MLP projection
        {"name": "linear, batch of 37", "op": "fp8_fwd", "m": 37, "n": 11008, "k": 4096, "fmt": "e4m3", "rows": "bf16"},
        # odd sizes: the last block of every axis is a short one
        {"name": "linear, ragged", "op": "fp8_fwd", "m": 333, "n": 1003, "k": 4112, "fmt": "e4m3", "rows": "bf16"},
        # 4096 prompt or training tokens, whose rows the norm in front left in 8 bits
        {"name": "linear, 4096 tokens", "op": "fp8_fwd", "m": 4096, "n": 11008, "k": 4096, "fmt": "e4m3",
         "rows": "fp8"},
        # gradient through the frozen down projection in training
        {"name": "linear gradient, 4096 tokens", "op": "fp8_bwd", "m": 4096, "n": 4096, "k": 11008, "fmt": "e4m3",
         "rows": "bf16"},
        # the norm in front of a projection for one generated token
        {"name": "norm, one token", "op": "norm", "rows": 1, "d": 4096, "res": True, "out": "e4m3"},
        # the same for a prompt of 4096 tokens and the wide hidden size
        {"name": "norm, 4096 tokens", "op": "norm", "rows": 4096, "d": 8192, "res": True, "out": "e4m3"},
        # an odd width that no vector load divides, bf16 output, no residual
        {"name": "norm, ragged", "op": "norm", "rows": 777, "d": 4099, "res": False, "out": "bf16"},
        # training: gradients of the input and of the gain
        {"name": "norm gradient, 4096 tokens", "op": "norm_bwd", "rows": 4096, "d": 4096, "res": True},
        # rank-8 adapters on two projections of 32 layers: many small tensors
        {"name": "adamw, 128 small tensors", "op": "adamw", "tensors": "pairs", "count": 128, "size": 32768,
         "bits": 32},
        # tensors of odd lengths, from one value up
        {"name": "adamw, odd tensors in 8 bits", "op": "adamw", "tensors": "odd", "count": 9, "size": 70001,
         "bits": 8},
        # rank-64 adapters on all seven projections of 32 layers of a 7B-shaped stack
        {"name": "adamw, 448 tensors in 8 bits", "op": "adamw", "tensors": "stack", "count": 448, "size": 64,
         "bits": 8},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["fp8_fwd", "fp8_fwd", "fp8_bwd", "norm", "norm_bwd", "adamw"])
    if op in ("fp8_fwd", "fp8_bwd"):
        while True:
            m, n, k = _log(rng, 1, 4096), _log(rng, 64, 12000), 16 * _log(rng, 8, 700)
            if m * n * k <= 4096 * 11008 * 4096:
                break
        fmt = "e4m3" if op == "fp8_fwd" else rng.choice(["e4m3", "e5m2"])
        return {"op": op, "m": m, "n": n, "k": k, "fmt": fmt, "rows": rng.choice(["bf16", "fp8"])}
    if op in ("norm", "norm_bwd"):
        while True:
            rows, d = _log(rng, 1, 8192), _log(rng, 64, 16384)
            if rows * d <= 4096 * 8192:
                break
        if rng.random() < 0.6:
            d = max(64, d // 64 * 64)
        case = {"op": op, "rows": rows, "d": d, "res": rng.random() < 0.7}
        if op == "norm":
            case["out"] = rng.choice(["bf16", "e4m3"])
        return case
    kind = rng.choice(["pairs", "odd"])
    return {"op": op, "tensors": kind, "count": _log(rng, 1, 448), "size": _log(rng, 64, 300000),
            "bits": rng.choice([8, 32])}


def _sizes(case):
    """Lengths of the tensors of one optimizer group."""
    if case["tensors"] == "stack":
        r = case["size"]
        io = [(4096, 4096)] * 4 + [(4096, 11008)] * 2 + [(11008, 4096)]
        return [v for _ in range(case["count"] // 14) for i, o in io for v in (r * i, r * o)]
    if case["tensors"] == "odd":
        return [max(1, (case["size"] | 1) * i * i // case["count"] ** 2) for i in range(case["count"])]
    return [case["size"]] * case["count"]


def _up(v, b):
    return -(-v // b) * b


# ---------------------------------------------------------------- inputs
def _quantize_weight(w):
    n, k = w.shape
    wf = torch.zeros(_up(n, BLOCK), _up(k, BLOCK), device=w.device)
    wf[:n, :k] = w
    t = wf.view(_up(n, BLOCK) // BLOCK, BLOCK, _up(k, BLOCK) // BLOCK, BLOCK)
    amax = t.abs().amax(dim=(1, 3)).clamp_min(LEAST)
    codes = (t * (448.0 / amax)[:, None, :, None]).clamp(-448, 448).view(wf.shape)[:n, :k]
    return codes.contiguous().to(torch.float8_e4m3fn), amax / 448.0


def _activations(g, m, k):
    """Tokens with a few wide channels, as hidden states have."""
    x = torch.randn(m, k, generator=g, device="cuda")
    wide = torch.rand(k, generator=g, device="cuda") < 0.004
    return torch.where(wide, x * 12.0, x).to(torch.bfloat16)


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    s = {"case": case}
    if case["op"] in ("fp8_fwd", "fp8_bwd"):
        m, n, k = case["m"], case["n"], case["k"]
        s["codes"], s["scales"] = _quantize_weight(torch.randn(n, k, generator=g, device="cuda").mul_(0.02).bfloat16())
        if case["op"] == "fp8_fwd":
            s["x"] = _activations(g, m, k)
        else:
            # gradients: small, and of another size from token to token
            size = torch.exp(torch.randn(m, 1, generator=g, device="cuda")) * 1e-4
            s["x"] = (torch.randn(m, n, generator=g, device="cuda") * size).bfloat16()
        if case["rows"] == "fp8":
            # rows that an earlier call left in 8 bits, each padded to a multiple of 16 bytes
            codes, s["x_scales"] = _plain_rows(s["x"].float(), case["fmt"])
            wide = torch.zeros(m, _up(codes.shape[1], 16), device="cuda", dtype=torch.uint8)
            wide[:, :codes.shape[1]] = codes.view(torch.uint8)
            s["x_codes"] = wide.view(codes.dtype)[:, :codes.shape[1]]
            del s["x"]
    elif case["op"] in ("norm", "norm_bwd"):
        rows, d = case["rows"], case["d"]
        s["gamma"] = (1.0 + 0.2 * torch.randn(d, generator=g, device="cuda")).bfloat16()
        s["x"] = _activations(g, rows, d)
        s["res"] = _activations(g, rows, d) if case["res"] else None
        if case["op"] == "norm_bwd":
            s["rstd"] = torch.rsqrt(s["x"].float().square().mean(1) + NORM_EPS)
            s["dy"] = (torch.randn(rows, d, generator=g, device="cuda") * 1e-2).bfloat16()
    else:
        sizes = _sizes(case)
        starts = np.concatenate([[0], np.cumsum([_up(v, STATE_BLOCK) for v in sizes])]).tolist()
        total = starts[-1]
        cut = lambda flat: [flat[a:a + v] for a, v in zip(starts, sizes)]  # noqa: E731
        live = torch.zeros(total, dtype=torch.bool, device="cuda")
        for t in cut(live):
            t.fill_(True)
        # one flat buffer each, every tensor at a multiple of 256 values
        s["master"] = torch.randn(total, generator=g, device="cuda").mul_(0.02).mul_(live)
        s["param"] = s["master"].bfloat16()
        s["masters"], s["params"] = cut(s["master"]), cut(s["param"])
        noise = torch.randn(total, generator=g, device="cuda") * 1e-3
        s["grads"] = [v.clone() for v in cut(noise)]
        m = (torch.randn(total, generator=g, device="cuda") * 3e-4).mul_(live)
        r = ((0.4 + torch.rand(total, generator=g, device="cuda")) * 1e-3).mul_(live)
        if case["bits"] == 8:
            s["m"], s["m_scales"] = _plain_state(m, False)
            s["v"], s["v_scales"] = _plain_state(r, True)
        else:
            s["m"], s["v"], s["m_scales"], s["v_scales"] = m, r.square(), None, None
        if own:
            # the optimizer object that a program makes once
            import bit_nf4_quantized_06_b200 as q
            s["group"] = q.AdamWGroup(s["masters"], params=s["params"], bits=case["bits"], m=s["m"], v=s["v"],
                                      m_scales=s["m_scales"], v_scales=s["v_scales"])
    return s


# ---------------------------------------------------------------- plain forms
def _plain_rows(x, fmt):
    """Codes and scales of fp32 rows, one scale per 128 columns."""
    m, k = x.shape
    top = TOP[fmt]
    t = torch.nn.functional.pad(x, (0, _up(k, BLOCK) - k)).view(m, -1, BLOCK)
    amax = t.abs().amax(2).clamp_min(LEAST)
    codes = (t * (top / amax)[:, :, None]).clamp(-top, top).view(m, -1)[:, :k]
    return codes.to(FP8[fmt]).contiguous(), amax / top


def _plain_state(v, root):
    """e4m3 codes and scales by blocks of 256; a root above zero keeps a code above zero."""
    t = v.view(-1, STATE_BLOCK)
    amax = t.abs().amax(1).clamp_min(LEAST)
    c = (t * (448.0 / amax)[:, None]).clamp(-448, 448)
    if root:
        c = torch.where(t > 0, c.clamp_min(2.0 ** -9), c)
    return c.to(torch.float8_e4m3fn).view(-1), amax / 448.0


def _wide_rows(scales, k):
    return scales.repeat_interleave(BLOCK, 1)[:, :k]


def _wide_weight(scales, n, k):
    return _wide_rows(scales, k).repeat_interleave(BLOCK, 0)[:n]


def _plain_linear(s):
    case = s["case"]
    fwd = case["op"] == "fp8_fwd"
    codes, scales = (s["x_codes"], s["x_scales"]) if "x_codes" in s else _plain_rows(s["x"].float(), case["fmt"])
    x = codes.float() * _wide_rows(scales, codes.shape[1])
    w = s["codes"].float() * _wide_weight(s["scales"], case["n"], case["k"])
    return torch.matmul(x, w.t() if fwd else w).bfloat16()


def _plain_norm(s):
    h = s["x"] if s["res"] is None else (s["x"].float() + s["res"].float()).bfloat16()
    hf = h.float()
    rstd = torch.rsqrt(hf.square().mean(1) + NORM_EPS)
    y = hf * rstd[:, None] * s["gamma"].float()
    out = {"rstd": rstd}
    if s["res"] is not None:
        out["h"] = h
    if s["case"]["out"] == "bf16":
        out["y"] = y.bfloat16()
    else:
        out["codes"], out["scales"] = _plain_rows(y, s["case"]["out"])
    return out


def _plain_norm_bwd(s):
    h, dy, rstd = s["x"].float(), s["dy"].float(), s["rstd"][:, None]
    dyg = dy * s["gamma"].float()
    c = (dyg * h).mean(1, keepdim=True) * rstd.square()
    dx = (dyg - h * c) * rstd
    if s["res"] is not None:
        dx = dx + s["res"].float()
    return {"dx": dx.bfloat16(), "dgamma": (dy * (h * rstd)).sum(0)}


def _plain_adamw(s):
    pad = [_up(t.numel(), STATE_BLOCK) - t.numel() for t in s["grads"]]
    g = torch.cat([torch.nn.functional.pad(t, (0, p)) if p else t for t, p in zip(s["grads"], pad)])
    p = s["master"]
    if s["m_scales"] is not None:
        m = (s["m"].float().view(-1, STATE_BLOCK) * s["m_scales"][:, None]).view(-1)
        r = (s["v"].float().view(-1, STATE_BLOCK) * s["v_scales"][:, None]).view(-1)
        v = r * r
    else:
        m, v = s["m"], s["v"]
    m = m * BETA1 + g * (1.0 - BETA1)
    v = v * BETA2 + g * g * (1.0 - BETA2)
    r = torch.sqrt(v)
    denom = r * (1.0 / math.sqrt(1.0 - BETA2 ** STEP)) + EPS
    p.copy_(p * (1.0 - LR * DECAY) - (LR / (1.0 - BETA1 ** STEP)) * (m / denom))
    s["param"].copy_(p)
    if s["m_scales"] is not None:
        for_m, for_v = _plain_state(m, False), _plain_state(r, True)
        s["m"].copy_(for_m[0]), s["m_scales"].copy_(for_m[1])
        s["v"].copy_(for_v[0]), s["v_scales"].copy_(for_v[1])
    else:
        s["m"].copy_(m), s["v"].copy_(v)
    return _adamw_out(s)


def _adamw_out(s):
    out = {k: s[k] for k in ("master", "param", "m", "v")}
    if s["m_scales"] is not None:
        out["m_scales"], out["v_scales"] = s["m_scales"], s["v_scales"]
    return out


# ---------------------------------------------------------------- one pass
def run(state):
    s, op = state, state["case"]["op"]
    if not own:
        if op in ("fp8_fwd", "fp8_bwd"):
            return _plain_linear(s)
        if op == "norm":
            return _plain_norm(s)
        return _plain_norm_bwd(s) if op == "norm_bwd" else _plain_adamw(s)
    import bit_nf4_quantized_06_b200 as q
    if op in ("fp8_fwd", "fp8_bwd"):
        w = q.FP8Weight(s["codes"], s["scales"])
        x = q.FP8Rows(s["x_codes"], s["x_scales"]) if "x_codes" in s else s["x"]
        if op == "fp8_fwd":
            return q.qlora_fp8_linear_fwd(w, x)
        return q.qlora_fp8_linear_bwd(w, x, fmt=q.FP8_E5M2 if s["case"]["fmt"] == "e5m2" else q.FP8_E4M3)
    if op == "norm":
        fp8 = s["case"]["out"] != "bf16"
        y, h, rstd = q.qlora_rmsnorm_fwd(s["x"], s["gamma"], NORM_EPS, residual=s["res"], fp8=fp8)
        out = {"codes": y.codes, "scales": y.scales} if fp8 else {"y": y}
        if s["res"] is not None:
            out["h"] = h
        return {**out, "rstd": rstd}
    if op == "norm_bwd":
        dx, dgamma = q.qlora_rmsnorm_bwd(s["dy"], s["x"], s["gamma"], s["rstd"], dres=s["res"])
        return {"dx": dx, "dgamma": dgamma}
    q.qlora_adamw_multi(s["group"], s["grads"], STEP, lr=LR, betas=(BETA1, BETA2), eps=EPS, weight_decay=DECAY)
    return _adamw_out(s)


# ---------------------------------------------------------------- what a pass cannot do without
def work(case):
    if case["op"] in ("fp8_fwd", "fp8_bwd"):
        m, n, k = case["m"], case["n"], case["k"]
        a, o = (k, n) if case["op"] == "fp8_fwd" else (n, k)
        rows = 2 * m * a if case["rows"] == "bf16" else m * a + 4 * m * (_up(a, BLOCK) // BLOCK)
        scales = 4 * (_up(n, BLOCK) // BLOCK) * (_up(k, BLOCK) // BLOCK)
        return {"bytes": rows + n * k + scales + 2 * m * o, "flops": 2 * m * n * k}
    if case["op"] in ("norm", "norm_bwd"):
        rows, d = case["rows"], case["d"]
        if case["op"] == "norm_bwd":
            return {"bytes": rows * d * (6 + 2 * case["res"]) + 4 * rows + 6 * d, "flops": 10 * rows * d}
        out = 2 * d if case["out"] == "bf16" else d + 4 * (_up(d, BLOCK) // BLOCK)
        return {"bytes": rows * (2 * d + 4 * d * case["res"] + out + 4) + 2 * d, "flops": 6 * rows * d}
    values = sum(_sizes(case))
    return {"bytes": values * (30 if case["bits"] == 32 else 18) + (0 if case["bits"] == 32 else values // 16),
            "flops": 14 * values}


# ---------------------------------------------------------------- the definitions in fp64
def _exact_rows(v, top):
    """(unrounded code values, scales) in fp64, block by block."""
    cols = v.shape[1]
    values, scales = torch.empty_like(v), []
    for a in range(0, cols, 128):
        part = v[:, a:a + 128]
        scales.append(part.abs().max(dim=1).values.clamp_min(2.0 ** -100) / top)
        values[:, a:a + 128] = part / scales[-1][:, None]
    return values, torch.stack(scales, 1)


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] in ("fp8_fwd", "fp8_bwd"):
        if "x_codes" in s:
            x, sx = s["x_codes"].double(), s["x_scales"].double()
        else:
            top = 448.0 if case["fmt"] == "e4m3" else 57344.0
            x, sx = _exact_rows(s["x"].double(), top)
            x = x.float().clamp(-top, top).to(FP8[case["fmt"]]).double()
        x = x.contiguous()
        w = s["codes"].double()
        for j in range(sx.shape[1]):
            x[:, j * 128:(j + 1) * 128] *= sx[:, j:j + 1]
        for i in range(s["scales"].shape[0]):
            for j in range(s["scales"].shape[1]):
                w[i * 128:(i + 1) * 128, j * 128:(j + 1) * 128] *= s["scales"][i, j].double()
        return x @ w.t() if case["op"] == "fp8_fwd" else x @ w
    if case["op"] == "norm":
        h = s["x"].double()
        if s["res"] is not None:
            h = (s["x"].double() + s["res"].double()).bfloat16().double()
        rstd = 1.0 / ((h * h).sum(1) / h.shape[1] + NORM_EPS).sqrt()
        y = h * s["gamma"].double() * rstd[:, None]
        out = {"rstd": rstd}
        if s["res"] is not None:
            out["h"] = s["x"].double() + s["res"].double()
        if case["out"] == "bf16":
            out["y"] = y
        else:
            out["codes"], out["scales"] = _exact_rows(y, 448.0)
        return out
    if case["op"] == "norm_bwd":
        h, dy, gamma, rstd = (s[k].double() for k in ("x", "dy", "gamma", "rstd"))
        unit = h * rstd[:, None]
        up = dy * gamma
        dx = rstd[:, None] * (up - unit * (up * unit).sum(1, keepdim=True) / h.shape[1])
        return {"dx": dx if s["res"] is None else dx + s["res"].double(), "dgamma": (dy * unit).sum(0)}
    out = {"master": torch.zeros_like(s["master"], dtype=torch.float64)}
    m_new, r_new = torch.zeros_like(out["master"]), torch.zeros_like(out["master"])
    at = 0
    for p, g in zip(s["masters"], s["grads"]):
        n = p.numel()
        m, v = s["m"][at:at + n].double(), s["v"][at:at + n].double()
        if case["bits"] == 8:
            blocks = torch.arange(at, at + n, device=p.device) // 256
            m, v = m * s["m_scales"].double()[blocks], (v * s["v_scales"].double()[blocks]) ** 2
        g = g.double()
        m = BETA1 * m + (1 - BETA1) * g
        v = BETA2 * v + (1 - BETA2) * g ** 2
        m_hat, v_hat = m / (1 - BETA1 ** STEP), v / (1 - BETA2 ** STEP)
        out["master"][at:at + n] = p.double() - LR * DECAY * p.double() - LR * m_hat / (v_hat.sqrt() + EPS)
        m_new[at:at + n], r_new[at:at + n] = m, v.sqrt()
        at += -(-n // 256) * 256
    out["param"] = out["master"]
    if case["bits"] == 32:
        out["m"], out["v"] = m_new, r_new ** 2
        return out
    for name, v in (("m", m_new), ("v", r_new)):
        blocks = v.reshape(-1, 256)
        scale = blocks.abs().max(1).values.clamp_min(2.0 ** -100) / 448.0
        out[name], out[name + "_scales"] = (blocks / scale[:, None]).reshape(-1), scale
    return out
