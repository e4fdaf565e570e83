"""The dense operators around a routed-expert layer: what one call of each is measured on.

Three operators of a transformer block's dense half, forward and backward:

* layer norm over the rows a router and its experts read;
* the gated feed-forward product act(x w1^T) * (x w3^T) of a dense layer or a shared
  expert, one kernel for both projections, the activation and the product;
* the linear projection act(x w^T + bias) + residual that closes such a block.

`run` computes them in elementary torch operations in 32 bits, rounded once at the
end, or (with `own` true) through the library's calls.  A case's sizes: T rows, K input
columns, N output columns (layer norm has T and K only).
"""
import math

import torch

own = False

DEV = "cuda"
EPS = 1e-5
TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


def listed():
    def norm(name, way, T, K, dtype="bf16", grad="bf16"):
        return dict(name=name, op="norm", way=way, T=T, K=K, N=0, dtype=dtype, act="none", bias=True,
                    residual=False, save=way == "fwd" and T > 16, grad=grad)

    def gated(name, way, T, K, N, dtype="bf16", act="silu", save=False, grad="bf16"):
        return dict(name=name, op="gated", way=way, T=T, K=K, N=N, dtype=dtype, act=act, bias=False,
                    residual=False, save=save, grad=grad)

    def linear(name, way, T, K, N, dtype="bf16", act="none", bias=True, residual=False, save=False, grad="bf16"):
        return dict(name=name, op="linear", way=way, T=T, K=K, N=N, dtype=dtype, act=act, bias=bias,
                    residual=residual, save=save, grad=grad)

    return [
        # one decoding token's row before the router: the cost of a launch
        norm("norm_token", "fwd", 1, 4096),
        # a long prompt's (or a training step's) rows at the widest model width, statistics kept
        norm("norm_prompt", "fwd", 8192, 7168),
        # the same rows in training: dx and the sums over 8192 rows for the weight and the bias
        norm("norm_grad", "bwd", 8192, 7168),
        # a ragged fp32 batch with an odd width: rows that no wide load is aligned to
        norm("norm_grad_odd_f32", "bwd", 2049, 1021, dtype="f32", grad="f32"),
        # a decoding step of 8 sequences through a shared expert: the weights are read once
        gated("gated_decode", "fwd", 8, 7168, 2048),
        # the shared expert over a full prompt, inference
        gated("gated_prompt", "fwd", 8192, 7168, 2048),
        # a training step of a wide dense layer: gradients from the saved projections
        gated("gated_grad", "bwd", 4096, 2048, 8192),
        # a ragged training batch, sizes that end inside every tile
        gated("gated_train_ragged", "fwd", 1021, 1416, 2120, act="gelu_tanh", save=True),
        # one token's down projection added to the residual stream
        linear("linear_token", "fwd", 1, 2048, 7168, bias=False, residual=True),
        # a prompt's down projection with bias and residual
        linear("linear_prompt", "fwd", 8192, 2048, 7168, residual=True),
        # training through an activation: dx, dw and the bias gradient from the kept pre-activations
        linear("linear_grad", "bwd", 4096, 4096, 4096, act="gelu"),
        # a small fp32 layer with odd sizes and the activation in the epilogue
        linear("linear_odd_f32", "fwd", 515, 1001, 1777, dtype="f32", act="gelu", residual=True),
    ]


def _spread(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _width(rng, lo, hi):
    """Half of the widths are whole tiles, a quarter whole 16-byte chunks, the rest anything."""
    n, kind = _spread(rng, lo, hi), rng.random()
    step = 64 if kind < 0.5 else 8 if kind < 0.75 else 1
    return max(lo, n // step * step)


def draw(rng):
    op = rng.choice(["norm", "gated", "gated", "linear", "linear"])
    way = rng.choice(["fwd", "bwd"])
    dtype = "bf16" if rng.random() < 0.75 else "f32"
    T, K, N = _spread(rng, 1, 8192), _width(rng, 64, 7168), _width(rng, 64, 8192)
    if op != "norm":
        T = max(1, min(T, int(8192 * 7168 * 2048 / (K * N))))
    act = {"norm": ["none"], "gated": ["silu", "gelu", "gelu_tanh", "relu"],
           "linear": ["none", "none", "silu", "gelu", "gelu_tanh", "relu"]}[op]
    fwd = way == "fwd"
    return dict(op=op, way=way, T=T, K=K, N=0 if op == "norm" else N, dtype=dtype, act=rng.choice(act),
                bias=op != "gated" and rng.random() < 0.7,
                residual=op == "linear" and fwd and rng.random() < 0.6,
                save=fwd and rng.random() < 0.5,
                grad="f32" if dtype == "f32" or (not fwd and rng.random() < 0.3) else "bf16")


def prepare(case, seed):
    """Activations about N(0, 1), weights about N(0, 0.02^2), as a trained layer's; a norm's rows
    each with a mean and a scale of their own.  The backward passes get the statistics or the
    projections that a forward pass kept."""
    c, g = case, torch.Generator(device=DEV).manual_seed(seed)
    T, K, N, dt = c["T"], c["K"], c["N"], TYPES[c["dtype"]]

    def normal(*shape, std=1.0, mean=0.0, dtype=dt):
        return torch.empty(shape, device=DEV, dtype=torch.float32).normal_(mean, std, generator=g).to(dtype)

    s = {"case": dict(c), "kept": {}}
    if c["op"] == "norm":
        rows = normal(T, 2, dtype=torch.float32)
        s["x"] = (normal(T, K, dtype=torch.float32) * torch.exp2(rows[:, :1]) + rows[:, 1:]).to(dt)
        s["w"] = normal(K, std=0.1, mean=1.0)
        s["b"] = normal(K, std=0.1) if c["bias"] else None
        if c["way"] == "bwd":
            s["dy"] = normal(T, K)
            x = s["x"].float()
            s["mean"] = x.mean(1)
            s["rstd"] = torch.rsqrt((x - s["mean"][:, None]).square().mean(1) + EPS)
        return s
    s["x"] = normal(T, K)
    if c["op"] == "gated":
        s["w1"], s["w3"] = normal(N, K, std=0.02), normal(N, K, std=0.02)
        if c["way"] == "bwd":
            spread = 0.02 * math.sqrt(K)
            s["g"], s["u"], s["dh"] = normal(T, N, std=spread), normal(T, N, std=spread), normal(T, N)
        return s
    s["w"] = normal(N, K, std=0.02)
    s["bias"] = normal(N, std=0.1) if c["bias"] else None
    s["residual"] = normal(T, N) if c["residual"] else None
    if c["way"] == "bwd":
        s["dy"] = normal(T, N)
        s["z"] = normal(T, N, std=0.02 * math.sqrt(K)) if c["act"] != "none" else None
    return s


# ---- plain form

GELU_C = math.sqrt(2.0 / math.pi)


def _sigmoid(z):
    return 1.0 / (1.0 + torch.exp(-z))


def _act(z, act):
    if act == "none":
        return z
    if act == "relu":
        return torch.where(z > 0, z, torch.zeros_like(z))
    if act == "silu":
        return z * _sigmoid(z)
    if act == "gelu":
        return 0.5 * z * (1.0 + torch.erf(z * math.sqrt(0.5)))
    return 0.5 * z * (1.0 + torch.tanh(GELU_C * (z + 0.044715 * z * z * z)))


def _act_slope(z, act):
    if act == "none":
        return torch.ones_like(z)
    if act == "relu":
        return (z > 0).to(z.dtype)
    if act == "silu":
        s = _sigmoid(z)
        return s * (1.0 + z * (1.0 - s))
    if act == "gelu":
        return 0.5 * (1.0 + torch.erf(z * math.sqrt(0.5))) + z * torch.exp(-0.5 * z * z) / math.sqrt(2.0 * math.pi)
    t = torch.tanh(GELU_C * (z + 0.044715 * z * z * z))
    return 0.5 * (1.0 + t) + 0.5 * z * (1.0 - t * t) * GELU_C * (1.0 + 3.0 * 0.044715 * z * z)


def _plain(s):
    c = s["case"]
    dt, gt = TYPES[c["dtype"]], TYPES[c["grad"]]
    f = {k: v.float() for k, v in s.items() if isinstance(v, torch.Tensor)}
    x = f["x"]
    if c["op"] == "norm":
        if c["way"] == "fwd":
            mean = x.mean(1, keepdim=True)
            d = x - mean
            rstd = 1.0 / torch.sqrt((d * d).mean(1, keepdim=True) + EPS)
            y = d * rstd * f["w"]
            out = {"y": (y + f["b"] if c["bias"] else y).to(dt)}
            return dict(out, mean=mean[:, 0], rstd=rstd[:, 0]) if c["save"] else out
        xh = (x - f["mean"][:, None]) * f["rstd"][:, None]
        dy = f["dy"]
        e = dy * f["w"]
        dx = f["rstd"][:, None] * (e - e.mean(1, keepdim=True) - xh * (e * xh).mean(1, keepdim=True))
        out = {"dx": dx.to(dt), "dw": (dy * xh).sum(0).to(gt)}
        return dict(out, db=dy.sum(0).to(gt)) if c["bias"] else out
    if c["op"] == "gated":
        if c["way"] == "fwd":
            g, u = x @ f["w1"].T, x @ f["w3"].T
            out = {"h": (_act(g, c["act"]) * u).to(dt)}
            return dict(out, g=g.to(dt), u=u.to(dt)) if c["save"] else out
        dg = f["dh"] * f["u"] * _act_slope(f["g"], c["act"])
        du = f["dh"] * _act(f["g"], c["act"])
        return {"dx": (dg @ f["w1"] + du @ f["w3"]).to(dt), "dw1": (dg.T @ x).to(gt), "dw3": (du.T @ x).to(gt)}
    if c["way"] == "fwd":
        z = x @ f["w"].T
        if c["bias"]:
            z = z + f["bias"]
        y = _act(z, c["act"])
        out = {"y": (y + f["residual"] if c["residual"] else y).to(dt)}
        return dict(out, z=z.to(dt)) if c["save"] else out
    dz = f["dy"] * _act_slope(f["z"], c["act"]) if c["act"] != "none" else f["dy"]
    out = {"dx": (dz @ f["w"]).to(dt), "dw": (dz.T @ x).to(gt)}
    return dict(out, dbias=dz.sum(0).to(gt)) if c["bias"] else out


# ---- the library's calls

def _keep(s):
    """The shape, workspace and output buffers of this case, made at its first pass and kept, as
    a program that makes the call every step keeps them."""
    from routing_dispatch_expert_logits_amd import binding as B
    c, k = s["case"], s["kept"]
    T, K, N, dt, gt = c["T"], c["K"], c["N"], TYPES[c["dtype"]], TYPES[c["grad"]]

    def new(*shape, dtype=dt):
        return torch.empty(shape, device=DEV, dtype=dtype)

    k["B"] = B
    if c["op"] == "norm":
        k["shape"] = B.norm_shape(T, K, eps=EPS, dtype=c["dtype"], grad_dtype=c["grad"] if c["way"] == "bwd" else None)
        if c["way"] == "fwd":
            k["out"] = {"y": new(T, K)}
            if c["save"]:
                k["out"].update(mean=new(T, dtype=torch.float32), rstd=new(T, dtype=torch.float32))
        else:
            k["ws"] = new(B.norm_workspace_bytes(k["shape"]), dtype=torch.uint8)
            k["out"] = {"dx": new(T, K), "dw": new(K, dtype=gt)}
            if c["bias"]:
                k["out"]["db"] = new(K, dtype=gt)
        return k
    k["shape"] = B.dense_shape(T, K, N, dtype=c["dtype"], act=c["act"],
                               grad_dtype=c["grad"] if c["way"] == "bwd" else None)
    call = {("gated", "fwd"): B.MOE_CALL_GATED_FORWARD, ("gated", "bwd"): B.MOE_CALL_GATED_BACKWARD,
            ("linear", "fwd"): B.MOE_CALL_LINEAR_FORWARD, ("linear", "bwd"): B.MOE_CALL_LINEAR_BACKWARD}
    k["ws"] = new(B.dense_workspace_bytes(k["shape"], call[c["op"], c["way"]]), dtype=torch.uint8)
    if c["way"] == "fwd":
        names = ("h", "g", "u") if c["op"] == "gated" else ("y", "z")
        k["out"] = {n: new(T, N) for n in (names if c["save"] else names[:1])}
    elif c["op"] == "gated":
        k["out"] = {"dx": new(T, K), "dw1": new(N, K, dtype=gt), "dw3": new(N, K, dtype=gt)}
    else:
        k["out"] = {"dx": new(T, K), "dw": new(N, K, dtype=gt)}
        if c["bias"]:
            k["out"]["dbias"] = new(N, dtype=gt)
    return k


def _calls(s):
    k = s["kept"] or _keep(s)
    B, c, o, shape = k["B"], s["case"], k["out"], k["shape"]
    if c["op"] == "norm":
        if c["way"] == "fwd":
            B.layer_norm_forward(s["x"], s["w"], s["b"], o["y"], shape, mean=o.get("mean"), rstd=o.get("rstd"))
        else:
            B.layer_norm_backward(s["dy"], s["x"], s["w"], s["mean"], s["rstd"], o["dx"], o["dw"], o.get("db"),
                                  shape, k["ws"])
    elif c["op"] == "gated":
        if c["way"] == "fwd":
            B.gated_forward(s["x"], s["w1"], s["w3"], o["h"], shape, k["ws"], g=o.get("g"), u=o.get("u"))
        else:
            B.gated_backward(s["dh"], s["x"], s["w1"], s["w3"], s["g"], s["u"], o["dx"], o["dw1"], o["dw3"],
                             shape, k["ws"])
    elif c["way"] == "fwd":
        B.linear_forward(s["x"], s["w"], s["bias"], s["residual"], o["y"], shape, k["ws"], z=o.get("z"))
    else:
        B.linear_backward(s["dy"], s["x"], s["w"], s["z"], o["dx"], o["dw"], o.get("dbias"), shape, k["ws"])
    return o


def run(state):
    return _calls(state) if own else _plain(state)


def work(case):
    """Each input read once, each output written once, and the products' 2 T K N each."""
    c = case
    T, K, N = c["T"], c["K"], c["N"]
    e, ge = (2 if c["dtype"] == "bf16" else 4), (2 if c["grad"] == "bf16" else 4)
    if c["op"] == "norm":
        if c["way"] == "fwd":
            return {"bytes": e * (2 * T * K + (2 if c["bias"] else 1) * K) + (8 * T if c["save"] else 0),
                    "flops": 8 * T * K}
        return {"bytes": e * (3 * T * K + K) + 8 * T + ge * (2 if c["bias"] else 1) * K, "flops": 14 * T * K}
    if c["op"] == "gated":
        if c["way"] == "fwd":
            return {"bytes": e * (T * K + 2 * N * K + (3 if c["save"] else 1) * T * N), "flops": 4 * T * K * N}
        return {"bytes": e * (3 * T * N + 2 * T * K + 2 * N * K) + ge * 2 * N * K, "flops": 8 * T * K * N}
    if c["way"] == "fwd":
        more = (1 if c["save"] else 0) + (1 if c["residual"] else 0)
        return {"bytes": e * (T * K + N * K + (1 + more) * T * N + (N if c["bias"] else 0)), "flops": 2 * T * K * N}
    return {"bytes": e * ((2 if c["act"] != "none" else 1) * T * N + 2 * T * K + N * K) + ge * (N * K + (N if c["bias"] else 0)),
            "flops": 4 * T * K * N}


# ---- the definitions in 64 bits

def exact(case, seed):
    """From the definitions, with the activations' slopes by differentiation of their formulas
    through the normal distribution and the logistic function."""
    c, s = case, prepare(case, seed)
    v = {k: t.to(torch.float64) for k, t in s.items() if isinstance(t, torch.Tensor)}
    del s

    def value_and_slope(z):
        if c["act"] == "none":
            return z, 1.0
        if c["act"] == "relu":
            on = z.gt(0).double()
            return z * on, on
        if c["act"] == "silu":
            p = torch.special.expit(z)
            return z * p, p + z * p * torch.special.expit(-z)
        if c["act"] == "gelu":
            p = torch.special.ndtr(z)
            return z * p, p + z * torch.exp(-z * z / 2) / math.sqrt(2 * math.pi)
        # (1 + tanh q) / 2 = expit(2 q)
        q2 = math.sqrt(8 / math.pi) * (z + 0.044715 * z ** 3)
        p = torch.special.expit(q2)
        return z * p, p + z * p * torch.special.expit(-q2) * math.sqrt(8 / math.pi) * (1 + 0.134145 * z ** 2)

    if c["op"] == "norm":
        K = c["K"]
        if c["way"] == "fwd":
            var, mean = torch.var_mean(v["x"], dim=1, correction=0)
            scale = (var + EPS).pow(-0.5)
            y = torch.addcmul(v["b"], (v["x"] - mean.unsqueeze(1)).mul(scale.unsqueeze(1)), v["w"]) if c["bias"] else \
                (v["x"] - mean.unsqueeze(1)).mul(scale.unsqueeze(1)).mul(v["w"])
            return {"y": y, "mean": mean, "rstd": scale} if c["save"] else {"y": y}
        n = (v["x"] - v["mean"].unsqueeze(1)).mul(v["rstd"].unsqueeze(1))
        p = v["dy"].mul(v["w"])
        dots = torch.stack([p.sum(1), p.mul(n).sum(1)], 1) / K
        dx = (p - dots[:, :1] - n * dots[:, 1:]).mul(v["rstd"].unsqueeze(1))
        out = {"dx": dx, "dw": v["dy"].mul(n).sum(0)}
        if c["bias"]:
            out["db"] = v["dy"].sum(0)
        return out
    if c["op"] == "gated":
        if c["way"] == "fwd":
            both = torch.mm(v["x"], torch.cat([v["w1"], v["w3"]]).t())
            g, u = both.split(c["N"], dim=1)
            h = value_and_slope(g)[0] * u
            return {"h": h, "g": g.contiguous(), "u": u.contiguous()} if c["save"] else {"h": h}
        a, da = value_and_slope(v["g"])
        both = torch.cat([v["dh"] * v["u"] * da, v["dh"] * a], dim=1)
        dw1, dw3 = torch.mm(both.t(), v["x"]).split(c["N"], dim=0)
        return {"dx": torch.mm(both, torch.cat([v["w1"], v["w3"]])), "dw1": dw1, "dw3": dw3}
    if c["way"] == "fwd":
        z = torch.addmm(v["bias"], v["x"], v["w"].t()) if c["bias"] else torch.mm(v["x"], v["w"].t())
        y = value_and_slope(z)[0]
        if c["residual"]:
            y = y + v["residual"]
        return {"y": y, "z": z} if c["save"] else {"y": y}
    dz = v["dy"] * value_and_slope(v["z"])[1] if c["act"] != "none" else v["dy"]
    out = {"dx": torch.mm(dz, v["w"]), "dw": torch.mm(dz.t(), v["x"])}
    if c["bias"]:
        out["dbias"] = dz.sum(0)
    return out
