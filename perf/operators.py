"""The operators of a layer's training and serving step around the gated FFN, as they are measured:

* ``norm``: the norms before and after a block, fused with the block's gate, its residual scale and
  the residual sum (forward and backward);
* ``ffn``: the dense gated feed-forward block with a choice of activation (inference, down to one
  token, and a training step);
* ``adamw``: an AdamW step over many tensors, with fp32 or 8-bit states.

``run`` computes them in plain torch operations in 32 bits, or, with ``own`` set, through this
package's binding.  ``exact`` gives the same results from the definitions in 64 bits.
"""
import math

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
EPS = 1e-6
BETA1, BETA2, ADAM_EPS = 0.9, 0.95, 1e-8
LR, DECAY = 2e-4, 0.1
BLOCK = 256  # elements that share one scale of an 8-bit state


# ---------------------------------------------------------------------- cases --
def _norm(name, backward, T, d, y="bf16", r="f32", n="bf16", w="bf16", post=True, group=0,
          res=1.0, block=1.0):
    return {"name": name, "op": "norm", "backward": backward, "T": T, "d": d, "y": y, "r": r,
            "n": n, "w": w, "post": post, "group": group, "res": res, "block": block}


def _ffn(name, train, T, d, F, act):
    return {"name": name, "op": "ffn", "train": train, "T": T, "d": d, "F": F, "act": act}


def _adamw(name, sizes, bits, p, g, master):
    return {"name": name, "op": "adamw", "sizes": sizes, "bits": bits, "p": p, "g": g,
            "master": master}


def listed():
    M, V = 8192 * 2048, 2048  # a 2B layer's FFN matrix and norm vector
    return [
        # one decoded token between two layers of the 2B shape: the smallest call
        _norm("norm fwd 1 token", False, 1, 2048),
        # the prefill batch of the 2B shape, fp32 residual stream
        _norm("norm fwd 16384 tokens", False, 16384, 2048),
        # the training batch of the 2B shape, one gate vector (a learned per-channel scale)
        _norm("norm bwd 8192 tokens", True, 8192, 2048, group=8192, block=0.5),
        # ragged: 5 sequences of up to 700 tokens with a gate row each, bf16 residual stream, odd width
        _norm("norm bwd 5 gated sequences", True, 3301, 1000, r="bf16", group=700, res=0.9),
        # one decoded token, 2B weights: bound by reading the weights once
        _ffn("ffn fwd 1 token", False, 1, 2048, 8192, "silu"),
        # a decoding batch of odd size
        _ffn("ffn fwd 37 tokens", False, 37, 2048, 8192, "gelu"),
        # the prefill batch of the 2B shape
        _ffn("ffn fwd 16384 tokens", False, 16384, 2048, 8192, "silu"),
        # ragged training step: a part-filled batch on the 0.5B shape
        _ffn("ffn step 1003 tokens", True, 1003, 1024, 4096, "gelu_tanh"),
        # the training batch of the 2B shape
        _ffn("ffn step 8192 tokens", True, 8192, 2048, 8192, "silu"),
        # a few norm vectors and gates: many tensors, hardly any work
        _adamw("adamw 32 12 vectors", ",".join(["2048"] * 9 + ["1024", "1000", "1"]), 32, "f32",
               "f32", False),
        # a 2B layer: three FFN matrices and three vectors; bf16 weights, fp32 masters and gradients
        _adamw("adamw 32 2B layer", "%d,%d,%d,%d,%d,%d" % (M, M, M, V, V, V), 32, "bf16", "f32",
               True),
        # the same layer with 8-bit states, and bf16 gradients
        _adamw("adamw 8 2B layer", "%d,%d,%d,%d,%d,%d" % (M, M, M, V, V, V + 1), 8, "bf16", "bf16",
               True),
    ]


def _log(rng, lo, hi):
    return min(hi, max(lo, int(math.exp(rng.uniform(math.log(lo), math.log(hi + 1))))))


def draw(rng):
    op = rng.choice(["norm", "ffn", "adamw"])
    if op == "norm":
        backward = rng.random() < 0.5
        T = _log(rng, 1, 8192 if backward else 16384)
        d = 8 * _log(rng, 8, 256)
        group = rng.choice([0, T, _log(rng, 1, T)])
        r = rng.choice(["f32", "bf16"])
        c = _norm("", backward, T, d, y=rng.choice(["f32", "bf16"]), r=r, n="bf16",
                  w=rng.choice(["f32", "bf16"]), post=rng.random() < 0.7, group=group,
                  res=rng.choice([1.0, 0.9]), block=rng.choice([1.0, 0.5]))
    elif op == "ffn":
        train = rng.random() < 0.5
        T = _log(rng, 1, 8192 if train else 16384)
        c = _ffn("", train, T, 8 * rng.randint(16, 256), 8 * rng.randint(32, 1024),
                 rng.choice(["relu", "silu", "gelu", "gelu_tanh"]))
    else:
        bits = rng.choice([8, 32])
        sizes = [_log(rng, 1, 4 << 20) for _ in range(rng.randint(1, 12))]
        p = rng.choice(["f32", "bf16"])
        c = _adamw("", ",".join(str(s) for s in sizes), bits, p, rng.choice(["f32", "bf16"]),
                   p == "bf16" and rng.random() < 0.7)
    del c["name"]
    return c


# -------------------------------------------------------------------- prepare --
class _Normal:
    def __init__(self, seed):
        self.g = torch.Generator(device="cuda")
        self.g.manual_seed(int(seed))

    def __call__(self, *shape, scale=1.0, dtype=torch.float32):
        return (torch.randn(*shape, generator=self.g, device="cuda") * scale).to(dtype)

    def uniform(self, *shape):
        return torch.rand(*shape, generator=self.g, device="cuda")


def _prepare_norm(c, normal):
    T, d = c["T"], c["d"]
    yt, rt, nt, wt = (DTYPES[c[k]] for k in ("y", "r", "n", "w"))
    groups = -(-T // c["group"]) if c["group"] else 0
    s = {"y": normal(T, d, dtype=yt), "w_pre": (1 + normal(d, scale=0.1)).to(wt),
         "w_post": (1 + normal(d, scale=0.1)).to(wt) if c["post"] else None,
         "gate": normal(groups, d, scale=0.5, dtype=wt) if groups else None}
    r = normal(T, d, scale=2.0, dtype=rt)

    def empty(dtype):
        return torch.empty((T, d), dtype=dtype, device="cuda")

    if not c["backward"]:
        return {**s, "r": r, "r_out": empty(rt), "n_out": empty(nt)}
    # what the forward leaves behind: the new residual stream and the rows' inverse norms
    s.update(r_out=r, rstd_pre=1 / torch.sqrt(r.float().square().mean(1) + EPS),
             rstd_post=1 / torch.sqrt(s["y"].float().square().mean(1) + EPS) if c["post"] else None,
             dn=normal(T, d, dtype=nt), dr_out=normal(T, d, dtype=rt), dy=empty(yt), dr=empty(rt),
             dw_pre=torch.empty(d, device="cuda"),
             dw_post=torch.empty(d, device="cuda") if c["post"] else None,
             dgate=torch.empty((groups, d), device="cuda") if groups else None)
    if own:
        from activation_sparse_transformer_tma_b200 import twell
        s["ws"] = twell.norm_residual_backward_workspace(T, d, c["group"])
    return s


def _prepare_ffn(c, normal):
    T, d, F = c["T"], c["d"], c["F"]
    bf16 = torch.bfloat16

    def empty(*shape):
        return torch.empty(shape, dtype=bf16, device="cuda")

    s = {"x": normal(T, d, dtype=bf16), "Wg_t": normal(F, d, scale=d ** -0.5, dtype=bf16),
         "Wu_t": normal(F, d, scale=d ** -0.5, dtype=bf16),
         "Wd": normal(F, d, scale=F ** -0.5, dtype=bf16), "y": empty(T, d)}
    if c["train"]:
        s.update(dy=normal(T, d, dtype=bf16), z=empty(T, F), u=empty(T, F), dx=empty(T, d),
                 dWg_t=empty(F, d), dWu_t=empty(F, d), dWd=empty(F, d))
    if own:
        from activation_sparse_transformer_tma_b200 import twell
        s["status"] = torch.zeros(1, dtype=torch.int32, device="cuda")
        s["ws"] = twell.gated_ffn_workspace(T, d, F, training=c["train"])
    return s


def _prepare_adamw(c, normal):
    tensors = []
    for n in (int(v) for v in c["sizes"].split(",")):
        master = normal(n, scale=0.02)
        t = {"p": master.to(DTYPES[c["p"]]), "master": master if c["master"] else None,
             "g": normal(n, scale=1e-3, dtype=DTYPES[c["g"]])}
        m, v = normal(n, scale=3e-4), 1e-6 * (0.5 + normal.uniform(n))
        if c["bits"] == 32:
            t.update(m=m, v=v, m_scale=None, v_scale=None, m_values=None, v_values=None)
        else:
            # codes of the laws in _from_codes, and one scale for each block
            nb = -(-n // BLOCK)
            full = torch.zeros(2, nb * BLOCK, device="cuda")
            full[0, :n], full[1, :n] = m, v.sqrt()
            full = full.view(2, nb, BLOCK)
            top = full.abs().amax(2)
            ratio = (full.abs() / top.unsqueeze(2)).sqrt()
            t.update(m=(full[0].sign() * (ratio[0] * 127).round()).to(torch.int8).view(-1)[:n].clone(),
                     v=(ratio[1] * 255).round().to(torch.uint8).view(-1)[:n].clone(),
                     m_scale=top[0] / 127 ** 2, v_scale=top[1] / 255 ** 2,
                     m_values=torch.empty(n, dtype=torch.bfloat16, device="cuda"),
                     v_values=torch.empty(n, dtype=torch.bfloat16, device="cuda"))
        tensors.append(t)
    s = {"tensors": tensors, "step": 100}
    if own:
        from activation_sparse_transformer_tma_b200 import twell
        s["plan"] = twell.AdamWTensors([dict(t, weight_decay=DECAY) for t in tensors])
    return s


def prepare(case, seed):
    make = {"norm": _prepare_norm, "ffn": _prepare_ffn, "adamw": _prepare_adamw}[case["op"]]
    s = make(case, _Normal(seed))
    s["case"] = dict(case)
    return s


# ------------------------------------------------------------------------ run --
def _rows(gate, group, T):
    """The gate row of each token."""
    return 1.0 if gate is None else gate.float()[torch.arange(T, device="cuda") // group]


def _plain_norm_forward(c, s):
    y, r = s["y"].float(), s["r"].float()
    if c["post"]:
        y = y * torch.rsqrt(y.square().mean(1, keepdim=True) + EPS) * s["w_post"].float()
    r = c["res"] * r + c["block"] * (_rows(s["gate"], c["group"], c["T"]) * y)
    n = r * torch.rsqrt(r.square().mean(1, keepdim=True) + EPS) * s["w_pre"].float()
    return {"r": r.to(s["r"].dtype), "n": n.to(DTYPES[c["n"]])}


def _plain_norm_backward(c, s):
    T = c["T"]
    dn, y = s["dn"].float(), s["y"].float()
    rstd = s["rstd_pre"].unsqueeze(1)
    rh = s["r_out"].float() * rstd
    e = dn * s["w_pre"].float()
    g = s["dr_out"].float() + rstd * (e - rh * (e * rh).mean(1, keepdim=True))
    out = {"dw_pre": (dn * rh).sum(0), "dr": (c["res"] * g).to(s["r_out"].dtype)}
    k = c["block"] * (_rows(s["gate"], c["group"], T) * g)
    yh = y * s["rstd_post"].unsqueeze(1) if c["post"] else y
    if c["post"]:
        out["dw_post"] = (k * yh).sum(0)
        f = k * s["w_post"].float()
        out["dy"] = s["rstd_post"].unsqueeze(1) * (f - yh * (f * yh).mean(1, keepdim=True))
    else:
        out["dy"] = k
    out["dy"] = out["dy"].to(s["y"].dtype)
    if s["gate"] is not None:
        o = yh * s["w_post"].float() if c["post"] else yh
        rows = torch.arange(T, device="cuda") // c["group"]
        out["dgate"] = torch.zeros(s["gate"].shape, device="cuda").index_add_(
            0, rows, c["block"] * (g * o))
    return out


def _act(name, z):
    """The activation and its derivative."""
    if name == "relu":
        return z.clamp(min=0), (z > 0).to(z.dtype)
    if name == "silu":
        p = 1 / (1 + torch.exp(-z))
        return z * p, p * (1 + z * (1 - p))
    if name == "gelu":
        cdf = 0.5 * (1 + torch.erf(z * math.sqrt(0.5)))
        return z * cdf, cdf + z * torch.exp(-0.5 * z * z) / math.sqrt(2 * math.pi)
    k = math.sqrt(2 / math.pi)
    t = torch.tanh(k * (z + 0.044715 * z ** 3))
    return 0.5 * z * (1 + t), 0.5 * (1 + t) + 0.5 * z * (1 - t * t) * k * (1 + 0.134145 * z * z)


def _plain_ffn(c, s):
    x, Wg, Wu, Wd = (s[k].float() for k in ("x", "Wg_t", "Wu_t", "Wd"))
    bf16 = torch.bfloat16
    z, u = x @ Wg.T, x @ Wu.T
    a, da = _act(c["act"], z)
    h = a * u
    out = {"y": (h @ Wd).to(bf16)}
    if c["train"]:
        dy = s["dy"].float()
        dh = dy @ Wd.T
        du, dz = dh * a, dh * u * da
        out.update(dx=(du @ Wu + dz @ Wg).to(bf16), dWd=(h.T @ dy).to(bf16),
                   dWu_t=(du.T @ x).to(bf16), dWg_t=(dz.T @ x).to(bf16))
    return out


def _from_codes(codes, scale):
    """What 8-bit codes stand for: scale * c * |c| for m, and the same for sqrt(v)."""
    c = codes.float()
    return c * c.abs() * scale.repeat_interleave(BLOCK)[:c.numel()]


def _to_codes(values, most):
    """Codes and block scales of values; a value that is not zero keeps a code that is not zero
    where codes have no sign (most = 255)."""
    n = values.numel()
    full = torch.zeros(-(-n // BLOCK) * BLOCK, device="cuda")
    full[:n] = values
    full = full.view(-1, BLOCK)
    top = full.abs().amax(1, keepdim=True)
    ratio = torch.where(top > 0, full.abs() / torch.where(top > 0, top, 1.0), 0.0)
    code = (ratio.sqrt() * most).round()
    if most == 255:
        code = torch.where(full > 0, code.clamp(min=1), code)
    return (full.sign() * code).view(-1)[:n], top.view(-1) / most ** 2


def _plain_adamw(s, t):
    step = s["step"]
    g = t["g"].float()
    small = t["m_scale"] is not None
    m = _from_codes(t["m"], t["m_scale"]) if small else t["m"]
    v = _from_codes(t["v"], t["v_scale"]).square() if small else t["v"]
    m = BETA1 * m + (1 - BETA1) * g
    v = BETA2 * v + (1 - BETA2) * (g * g)
    p = (t["p"] if t["master"] is None else t["master"]).float()
    p = p * (1 - LR * DECAY) - (LR / (1 - BETA1 ** step)) * (
        m / (v.sqrt() * (1 - BETA2 ** step) ** -0.5 + ADAM_EPS))
    t["p"].copy_(p)
    if t["master"] is not None:
        t["master"].copy_(p)
    if not small:
        t["m"].copy_(m)
        t["v"].copy_(v)
        return
    for key, values, most in (("m", m, 127), ("v", v.sqrt(), 255)):
        code, scale = _to_codes(values, most)
        t[key].copy_(code)
        t[key + "_scale"].copy_(scale)
    t["m_values"].copy_(_from_codes(t["m"], t["m_scale"]))
    t["v_values"].copy_(_from_codes(t["v"], t["v_scale"]).square())


def _adamw_outputs(s):
    small = s["case"]["bits"] == 8
    keys = ("p", "master") + (("m_values", "v_values") if small else ("m", "v"))
    return [{k: t[k] for k in keys if t[k] is not None} for t in s["tensors"]]


def _run_own(c, s):
    from activation_sparse_transformer_tma_b200 import twell
    if c["op"] == "norm" and not c["backward"]:
        twell.norm_residual_forward(s["y"], s["r"], s["w_post"], s["gate"], s["w_pre"], s["r_out"],
                                    s["n_out"], gate_group=c["group"], res_scale=c["res"],
                                    block_scale=c["block"], eps=EPS)
        return {"r": s["r_out"], "n": s["n_out"]}
    if c["op"] == "norm":
        twell.norm_residual_backward(s["dn"], s["dr_out"], s["y"], s["r_out"], s["w_post"],
                                     s["gate"], s["w_pre"], s["rstd_post"], s["rstd_pre"], s["dy"],
                                     s["dr"], s["dw_post"], s["dgate"], s["dw_pre"], s["ws"],
                                     gate_group=c["group"], res_scale=c["res"],
                                     block_scale=c["block"])
        return {k: s[k] for k in ("dw_pre", "dr", "dw_post", "dy", "dgate") if s[k] is not None}
    if c["op"] == "ffn":
        twell.gated_ffn_forward(s["x"], s["Wg_t"], s["Wu_t"], s["Wd"], c["act"], s["y"], s["ws"],
                                z=s.get("z"), u=s.get("u"), dev_status=s["status"])
        if not c["train"]:
            return {"y": s["y"]}
        twell.gated_ffn_backward(s["x"], s["dy"], s["Wg_t"], s["Wu_t"], s["Wd"], c["act"], s["z"],
                                 s["u"], s["dx"], s["dWg_t"], s["dWu_t"], s["dWd"], s["ws"],
                                 dev_status=s["status"])
        return {k: s[k] for k in ("y", "dx", "dWd", "dWu_t", "dWg_t")}
    twell.adamw_step(s["plan"], lr=LR, beta1=BETA1, beta2=BETA2, eps=ADAM_EPS, step=s["step"])
    s["step"] += 1
    return _adamw_outputs(s)


def run(state):
    c = state["case"]
    if own:
        return _run_own(c, state)
    if c["op"] == "norm":
        return (_plain_norm_backward if c["backward"] else _plain_norm_forward)(c, state)
    if c["op"] == "ffn":
        return _plain_ffn(c, state)
    for t in state["tensors"]:
        _plain_adamw(state, t)
    state["step"] += 1
    return _adamw_outputs(state)


# ----------------------------------------------------------------------- work --
def work(case):
    size = {"bf16": 2, "f32": 4}
    c = case
    if c["op"] == "norm":
        e, w = c["T"] * c["d"], size[c["w"]] * c["d"]
        groups = -(-c["T"] // c["group"]) if c["group"] else 0
        vectors = 1 + (1 if c["post"] else 0) + groups
        if not c["backward"]:
            return {"bytes": e * (size[c["y"]] + 2 * size[c["r"]] + size[c["n"]]) + vectors * w,
                    "flops": 10 * e}
        saved = 4 * c["T"] * (2 if c["post"] else 1)
        return {"bytes": e * (size[c["n"]] + 3 * size[c["r"]] + 2 * size[c["y"]]) + saved
                + vectors * (w + 4 * c["d"]), "flops": 20 * e}
    if c["op"] == "ffn":
        T, d, F = c["T"], c["d"], c["F"]
        if not c["train"]:
            return {"bytes": 2 * (2 * T * d + 3 * d * F), "flops": 6 * T * d * F}
        return {"bytes": 2 * (4 * T * d + 6 * d * F), "flops": 18 * T * d * F}
    n = sum(int(v) for v in c["sizes"].split(","))
    state = 16 if c["bits"] == 32 else 4 + 4  # codes read and written, and their values written
    return {"bytes": n * (size[c["g"]] + size[c["p"]] * (1 if c["master"] else 2)
                          + (8 if c["master"] else 0) + state), "flops": 15 * n}


# ---------------------------------------------------------------------- exact --
def _double(v):
    return None if v is None else v.double()


def _exact_norm(c, s):
    T, group = c["T"], c["group"]
    s = {k: _double(v) for k, v in s.items() if v is None or torch.is_tensor(v)}
    rows = torch.arange(T, device="cuda") // group if group else None

    def unit(v):
        return v / (v.pow(2).mean(dim=-1, keepdim=True) + EPS) ** 0.5

    if not c["backward"]:
        o = unit(s["y"]) * s["w_post"] if c["post"] else s["y"]
        r = c["res"] * s["r"] + c["block"] * (o if rows is None else s["gate"][rows] * o)
        return {"r": r, "n": unit(r) * s["w_pre"]}
    # the saved rows' inverse norms are inputs: the gradients of v -> v * rstd(v) at those
    q = s["rstd_pre"][:, None]
    e = s["dn"] * s["w_pre"]
    inner = (e * s["r_out"]).sum(-1, keepdim=True) / c["d"]
    g = s["dr_out"] + q * e - q ** 3 * inner * s["r_out"]
    out = {"dr": c["res"] * g, "dw_pre": torch.einsum("td,td,t->d", s["dn"], s["r_out"], s["rstd_pre"])}
    k = c["block"] * g if rows is None else c["block"] * s["gate"][rows] * g
    p = s["rstd_post"][:, None] if c["post"] else None
    o = s["y"]
    if c["post"]:
        out["dw_post"] = torch.einsum("td,td,t->d", k, s["y"], s["rstd_post"])
        f = k * s["w_post"]
        out["dy"] = p * f - p ** 3 * (f * s["y"]).sum(-1, keepdim=True) / c["d"] * s["y"]
        o = s["y"] * p * s["w_post"]
    else:
        out["dy"] = k
    if rows is not None:
        parts = (c["block"] * g * o).split(group)
        out["dgate"] = torch.stack([v.sum(0) for v in parts])
    return out


def _exact_ffn(c, s):
    x, Wg, Wu, Wd = (s[k].double().requires_grad_(c["train"]) for k in ("x", "Wg_t", "Wu_t", "Wd"))
    z = x @ Wg.T
    if c["act"] == "relu":
        a = torch.relu(z)
    elif c["act"] == "silu":
        a = z * torch.sigmoid(z)
    elif c["act"] == "gelu":
        a = z * torch.special.ndtr(z)
    else:
        a = z * torch.sigmoid(math.sqrt(8 / math.pi) * (z + 0.044715 * z.pow(3)))
    y = (a * (x @ Wu.T)) @ Wd
    if not c["train"]:
        return {"y": y}
    gx, gg, gu, gd = torch.autograd.grad(y, (x, Wg, Wu, Wd), s["dy"].double())
    return {"y": y.detach(), "dx": gx, "dWd": gd, "dWu_t": gu, "dWg_t": gg}


def _exact_adamw(s):
    out = []
    for t in s["tensors"]:
        n, g = t["g"].numel(), t["g"].double()
        small = t["m_scale"] is not None
        block = torch.arange(n, device="cuda") // BLOCK
        m, v = t["m"].double(), t["v"].double()
        if small:
            m = m * m.abs() * t["m_scale"].double()[block]
            v = (v.pow(2) * t["v_scale"].double()[block]).pow(2)
        m = m + (1 - BETA1) * (g - m)
        v = v + (1 - BETA2) * (g.pow(2) - v)
        p = (t["p"] if t["master"] is None else t["master"]).double()
        step = (m / (1 - BETA1 ** s["step"])) / ((v / (1 - BETA2 ** s["step"])).sqrt() + ADAM_EPS)
        p = p - LR * DECAY * p - LR * step
        got = {"p": p}
        if t["master"] is not None:
            got["master"] = p
        if not small:
            got.update(m=m, v=v)
        else:
            for key, x, most in (("m", m, 127), ("v", v.sqrt(), 255)):
                top = torch.zeros(int(block[-1]) + 1, dtype=torch.float64, device="cuda")
                top = top.scatter_reduce(0, block, x.abs(), "amax")[block].clamp(min=1e-300)
                code = torch.round(most * (x.abs() / top).sqrt())
                if key == "v":
                    code = torch.where(x > 0, code.clamp(min=1), code)
                x = x.sign() * top * (code / most).pow(2)
                got[key + "_values"] = x if key == "m" else x.pow(2)
        out.append(got)
    return out


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "norm":
        return _exact_norm(case, s)
    if case["op"] == "ffn":
        return _exact_ffn(case, s)
    return _exact_adamw(s)
