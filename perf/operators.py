"""Cases and plain forms of the operators around the window attention of a layer.

A layer of the network is  x1 = x + W_o attn(W_qkv LN(x)),  y = x1 + FFN(LN(x1)):
layer norm, matrix products with bias, activation and residual, and a gated
feed-forward block, each with its backward pass.  Feature maps are seen as
[rows][channels], rows = batch * height * width.

  layer norm    mu = mean_c x, v = mean_c (x - mu)^2, r = 1 / sqrt(v + eps),
                xh = (x - mu) r,  y = gamma xh + beta
     backward   g = gamma dy,  dx = r (g - mean_c g - xh mean_c (g xh)) + dres,
                dgamma = sum_rows dy xh,  dbeta = sum_rows dy
  linear        z = x W^T + b,  y = act(z) + residual
     backward   dz = dy act'(z),  dx = dz W + dx_add,  dW = dz^T x,  db = sum_rows dz
  gated ffn     g = x Wg^T + bg,  u = x Wu^T + bu,  h = act(g) u,
                y = h Wo^T + bo + residual
     backward   dh = dy Wo,  dg = dh u act'(g),  du = dh act(g),
                dx = dg Wg + du Wu + dx_add,  dWg = dg^T x,  dWu = du^T x,
                dWo = dy^T h,  dbg, dbu, dbo = sum_rows dg, du, dy
  activations   gelu(z) = z Phi(z) (erf form),  silu(z) = z / (1 + e^-z)

Features, their gradients and the matrices are bf16 (layer norm also takes
fp32 features); biases, gamma, beta, statistics and their gradients fp32.
"""
import math

import torch

own = False

_EPS = 1e-5


def listed():
    return [
        # the normalisation of a 64 x 64 map of 3 heads: launch latency
        dict(name="norm_fwd_64x64_map", op="norm_fwd", rows=4096, channels=96, type="bf16"),
        # a batch of 8 maps of 192 x 192, 6 heads: a plain stream
        dict(name="norm_fwd_8_maps", op="norm_fwd", rows=294912, channels=192, type="bf16"),
        # its gradient in a training step, joined with the residual's
        dict(name="norm_bwd_4_maps", op="norm_bwd", rows=147456, channels=192, type="bf16"),
        # fp32 features, odd in both sizes
        dict(name="norm_bwd_f32_odd", op="norm_bwd", rows=9217, channels=333, type="fp32"),
        # one token through a wide projection: the weights' bytes and latency
        dict(name="linear_fwd_one_row", op="linear_fwd", rows=1, k=1024, n=4096, act="gelu",
             residual=False),
        # queries, keys and values of four 192 x 192 maps
        dict(name="linear_fwd_qkv", op="linear_fwd", rows=147456, k=192, n=576, act="none",
             residual=False),
        # ragged in every size, with everything in the epilogue
        dict(name="linear_fwd_ragged", op="linear_fwd", rows=5003, k=1032, n=2056, act="gelu",
             residual=True),
        # the gradient of queries, keys and values
        dict(name="linear_bwd_qkv", op="linear_bwd", rows=147456, k=192, n=576, act="none",
             residual=False),
        # ragged, through the activation, dx joined with another path's
        dict(name="linear_bwd_ragged", op="linear_bwd", rows=3001, k=520, n=1480, act="gelu",
             residual=True),
        # the feed-forward block of four 192 x 192 maps
        dict(name="ffn_fwd_4_maps", op="ffn_fwd", rows=147456, channels=192, hidden=384,
             act="silu", residual=True),
        # a wide block: bound by the tensor cores
        dict(name="ffn_fwd_wide", op="ffn_fwd", rows=8192, channels=1024, hidden=2816,
             act="gelu", residual=False),
        # the block's gradient in a training step of four 192 x 192 maps
        dict(name="ffn_bwd_4_maps", op="ffn_bwd", rows=147456, channels=192, hidden=384,
             act="silu", residual=False),
    ]


_MOST_FLOPS, _MOST_BYTES = 1.4e11, 2.2e8


def draw(rng):
    def spread(low, high, step=1):
        v = int(round(math.exp(rng.uniform(math.log(low), math.log(high))) / step)) * step
        return max(step * -(-low // step), v)

    op = rng.choice(["norm_fwd", "norm_bwd", "linear_fwd", "linear_bwd", "ffn_fwd", "ffn_bwd"])
    case = dict(op=op, rows=spread(1, 200000))
    if op.startswith("norm"):
        case.update(channels=spread(3, 4096), type=rng.choice(["bf16", "fp32"]))
    elif op.startswith("linear"):
        case.update(k=spread(16, 4096, 8), n=spread(16, 4096, 8),
                    act=rng.choice(["none", "gelu", "silu"]), residual=rng.random() < 0.5)
    else:
        case.update(channels=spread(16, 1024, 8), hidden=spread(16, 2816, 8),
                    act=rng.choice(["gelu", "silu"]), residual=rng.random() < 0.5)
    while case["rows"] > 1:
        w = work(case)
        if w["flops"] <= _MOST_FLOPS and w["bytes"] <= _MOST_BYTES:
            break
        case["rows"] = case["rows"] * 2 // 3
    return case


def _tensors(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)

    def normal(*shape, std=1.0, dtype=torch.bfloat16):
        return (torch.randn(shape, generator=g, device="cuda") * std).to(dtype)

    op, f32 = case["op"], torch.float32
    if op.startswith("norm"):
        rows, c = case["rows"], case["channels"]
        dtype = torch.bfloat16 if case["type"] == "bf16" else f32
        # features with a channel's own offset and scale, as a residual stream has
        x = normal(rows, c, dtype=f32) * (1 + normal(c, std=0.3, dtype=f32)) + normal(c, std=0.5, dtype=f32)
        t = dict(x=x.to(dtype), gamma=1 + normal(c, std=0.2, dtype=f32),
                 beta=normal(c, std=0.2, dtype=f32))
        if op == "norm_bwd":
            xd = t["x"].double()
            mean = xd.mean(1)
            rstd = ((xd - mean[:, None]).square().mean(1) + _EPS).rsqrt()
            t.update(mean=mean.float(), rstd=rstd.float(), dy=normal(rows, c, dtype=dtype),
                     dres=normal(rows, c, dtype=dtype))
        return t
    if op.startswith("linear"):
        rows, k, n = case["rows"], case["k"], case["n"]
        t = dict(x=normal(rows, k), w=normal(n, k, std=k ** -0.5))
        if op == "linear_fwd":
            t["bias"] = normal(n, std=0.1, dtype=f32)
            if case["residual"]:
                t["residual"] = normal(rows, n)
        else:
            t["dy"] = normal(rows, n)
            if case["act"] != "none":
                t["pre"] = normal(rows, n)
            if case["residual"]:
                t["dx_add"] = normal(rows, k)
        return t
    rows, c, hid = case["rows"], case["channels"], case["hidden"]
    t = dict(x=normal(rows, c), w_in=normal(2, hid, c, std=c ** -0.5),
             b_in=normal(2, hid, std=0.1, dtype=f32), w_out=normal(c, hid, std=hid ** -0.5),
             b_out=normal(c, std=0.1, dtype=f32))
    if op == "ffn_bwd":
        t["dy"] = normal(rows, c)
    if case["residual"]:
        t["residual" if op == "ffn_fwd" else "dx_add"] = normal(rows, c)
    return t


def prepare(case, seed):
    return dict(case=case, **_tensors(case, seed))


# ------------------------------------------------------------------ plain form

def _act(z, name):
    if name == "gelu":
        return z * (0.5 * (1 + torch.erf(z * math.sqrt(0.5))))
    if name == "silu":
        return z / (1 + torch.exp(-z))
    return z


def _act_grad(z, name):
    if name == "gelu":
        return (0.5 * (1 + torch.erf(z * math.sqrt(0.5)))
                + z * torch.exp(-0.5 * z * z) * (1 / math.sqrt(2 * math.pi)))
    if name == "silu":
        s = 1 / (1 + torch.exp(-z))
        return s * (1 + z * (1 - s))
    return torch.ones_like(z)


def _plain(s):
    case, op = s["case"], s["case"]["op"]
    f = {n: v.float() for n, v in s.items() if isinstance(v, torch.Tensor)}
    x = f["x"]
    if op == "norm_fwd":
        mean = x.mean(1)
        d = x - mean[:, None]
        rstd = 1 / torch.sqrt((d * d).mean(1) + _EPS)
        y = d * rstd[:, None] * f["gamma"] + f["beta"]
        return dict(y=y.to(s["x"].dtype), mean=mean, rstd=rstd)
    if op == "norm_bwd":
        xh = (x - f["mean"][:, None]) * f["rstd"][:, None]
        g = f["dy"] * f["gamma"]
        dx = f["rstd"][:, None] * (g - g.mean(1, keepdim=True) - xh * (g * xh).mean(1, keepdim=True))
        return dict(dx=(dx + f["dres"]).to(s["x"].dtype), dgamma=(f["dy"] * xh).sum(0),
                    dbeta=f["dy"].sum(0))
    bf = torch.bfloat16
    if op == "linear_fwd":
        y = _act(x @ f["w"].t() + f["bias"], case["act"])
        if "residual" in f:
            y = y + f["residual"]
        return dict(y=y.to(bf))
    if op == "linear_bwd":
        dz = f["dy"] * _act_grad(f["pre"], case["act"]) if "pre" in f else f["dy"]
        dx = dz @ f["w"]
        if "dx_add" in f:
            dx = dx + f["dx_add"]
        dw = dz.t() @ x
        return dict(dx=dx.to(bf), dw=dw if case["act"] == "none" else dw.to(bf), db=dz.sum(0))
    g = x @ f["w_in"][0].t() + f["b_in"][0]
    u = x @ f["w_in"][1].t() + f["b_in"][1]
    a = _act(g, case["act"])
    if op == "ffn_fwd":
        y = (a * u) @ f["w_out"].t() + f["b_out"]
        if "residual" in f:
            y = y + f["residual"]
        return dict(y=y.to(bf))
    dy = f["dy"]
    dh = dy @ f["w_out"]
    dg, du = dh * u * _act_grad(g, case["act"]), dh * a
    dx = dg @ f["w_in"][0] + du @ f["w_in"][1]
    if "dx_add" in f:
        dx = dx + f["dx_add"]
    return dict(dx=dx.to(bf), dw_in=torch.stack([dg.t() @ x, du.t() @ x]).to(bf),
                db_in=torch.stack([dg.sum(0), du.sum(0)]), dw_out=(dy.t() @ (a * u)).to(bf),
                db_out=dy.sum(0))


# ------------------------------------------------------------------ the framework's calls

def _own(s):
    import windowed_attention_implicit_b200 as rib

    case, op = s["case"], s["case"]["op"]
    if op == "norm_fwd":
        y, mean, rstd = rib.rib_layer_norm_fwd(s["x"], s["gamma"], s["beta"], eps=_EPS)
        return dict(y=y, mean=mean, rstd=rstd)
    if op == "norm_bwd":
        return rib.rib_layer_norm_bwd(s["x"], s["dy"], s["mean"], s["rstd"], s["gamma"],
                                      dres=s["dres"])
    if op == "linear_fwd":
        y, _ = rib.rib_linear_fwd(s["x"], s["w"], s["bias"], act=case["act"],
                                  residual=s.get("residual"))
        return dict(y=y)
    if op == "linear_bwd":
        # through an activation dz is rounded to bf16 before the products, so
        # the weight's gradient is asked for in the weight's own type
        return rib.rib_linear_bwd(s["x"], s["w"], s["dy"], act=case["act"], pre=s.get("pre"),
                                  dx_add=s.get("dx_add"),
                                  dw_dtype=torch.float32 if case["act"] == "none" else torch.bfloat16)
    ffn = rib.GatedFfn(s["w_in"], s["b_in"], s["w_out"], s["b_out"])
    if op == "ffn_fwd":
        return dict(y=rib.rib_gated_ffn_fwd(s["x"], ffn, act=case["act"], residual=s.get("residual")))
    return rib.rib_gated_ffn_bwd(s["x"], ffn, s["dy"], act=case["act"], dx_add=s.get("dx_add"),
                                 dw_dtype=torch.bfloat16)


def run(state):
    return _own(state) if own else _plain(state)


# ------------------------------------------------------------------ what it cannot do without

def work(case):
    op, rows = case["op"], case["rows"]
    if op.startswith("norm"):
        c, e = case["channels"], 2 if case["type"] == "bf16" else 4
        if op == "norm_fwd":
            return dict(bytes=2 * e * rows * c + 8 * rows + 8 * c, flops=8 * rows * c)
        return dict(bytes=4 * e * rows * c + 8 * rows + 12 * c, flops=14 * rows * c)
    if op.startswith("linear"):
        k, n = case["k"], case["n"]
        if op == "linear_fwd":
            maps = rows * k + rows * n * (2 if case["residual"] else 1)
            return dict(bytes=2 * (maps + n * k) + 4 * n, flops=2 * rows * n * k)
        through = case["act"] != "none"
        maps = rows * n * (2 if through else 1) + rows * k * (3 if case["residual"] else 2)
        return dict(bytes=2 * (maps + n * k) + (2 if through else 4) * n * k + 4 * n,
                    flops=4 * rows * n * k)
    c, hid = case["channels"], case["hidden"]
    maps = rows * c * (3 if case["residual"] else 2)
    if op == "ffn_fwd":
        return dict(bytes=2 * (maps + 3 * hid * c) + 4 * (2 * hid + c), flops=6 * rows * c * hid)
    return dict(bytes=2 * (maps + rows * c + 6 * hid * c) + 4 * (4 * hid + c),
                flops=16 * rows * c * hid)


# ------------------------------------------------------------------ the definition in 64 bits

def exact(case, seed):
    t = _tensors(case, seed)
    d = {n: v.to(torch.float64) for n, v in t.items()}
    op, act = case["op"], case.get("act")

    def phi(z):   # the normal distribution function
        return torch.special.erfc(-z * 2 ** -0.5) * 0.5

    def value(z):
        if act == "gelu":
            return z * phi(z)
        return z * torch.special.expit(z) if act == "silu" else z

    def slope(z):
        if act == "gelu":
            return phi(z) + z * torch.exp(-z.square() / 2) * (2 * math.pi) ** -0.5
        if act == "silu":
            p = torch.special.expit(z)
            return p + z * p * torch.special.expit(-z)
        return torch.ones_like(z)

    if op.startswith("norm"):
        x, c = d["x"], case["channels"]
        if op == "norm_fwd":
            mean = x.sum(1) / c
            rstd = ((x - mean[:, None]).pow(2).sum(1) / c + _EPS).pow(-0.5)
            y = torch.addcmul(d["beta"], (x - mean[:, None]) * rstd[:, None], d["gamma"])
            return dict(y=y, mean=mean, rstd=rstd)
        r = d["rstd"][:, None]
        xh = (x - d["mean"][:, None]) * r
        wdy = d["dy"] * d["gamma"]
        along = torch.einsum("rc,rc->r", wdy, xh)[:, None] / c
        dx = d["dres"] + (wdy - wdy.sum(1, keepdim=True) / c - along * xh) * r
        return dict(dx=dx, dgamma=torch.einsum("rc,rc->c", d["dy"], xh), dbeta=d["dy"].sum(0))
    if op == "linear_fwd":
        y = value(torch.addmm(d["bias"], d["x"], d["w"].t()))
        return dict(y=y + d["residual"] if "residual" in d else y)
    if op == "linear_bwd":
        dz = d["dy"] * slope(d["pre"]) if "pre" in d else d["dy"]
        dx = torch.einsum("rn,nk->rk", dz, d["w"])
        return dict(dx=dx + d["dx_add"] if "dx_add" in d else dx,
                    dw=torch.einsum("rn,rk->nk", dz, d["x"]), db=dz.sum(0))
    gu = torch.einsum("rc,ihc->irh", d["x"], d["w_in"]) + d["b_in"][:, None]
    if op == "ffn_fwd":
        y = torch.addmm(d["b_out"], value(gu[0]) * gu[1], d["w_out"].t())
        return dict(y=y + d["residual"] if "residual" in d else y)
    dh = torch.einsum("rc,ch->rh", d["dy"], d["w_out"])
    dgu = torch.stack([dh * gu[1] * slope(gu[0]), dh * value(gu[0])])
    dx = torch.einsum("irh,ihc->rc", dgu, d["w_in"])
    return dict(dx=dx + d["dx_add"] if "dx_add" in d else dx,
                dw_in=torch.einsum("irh,rc->ihc", dgu, d["x"]), db_in=dgu.sum(1),
                dw_out=torch.einsum("rc,rh->ch", d["dy"], value(gu[0]) * gu[1]),
                db_out=d["dy"].sum(0))
