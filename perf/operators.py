"""The training pass of the MoE block, operator by operator: what is run, on what, and what it costs.

The operators are the layer norm in front of the block (``moe_layer_norm`` and its backward),
the gradients of the token sort and the weighted return (``moe_permute_backward``,
``moe_combine_backward``), of the router (``moe_route_backward``) and of the grouped SwiGLU
experts (``moe_grouped_swiglu_backward``).

``listed()`` and ``draw()`` give cases, ``prepare()`` the inputs a program has in hand, ``run()``
one pass through the operator: with ``own`` false its plain form in elementary torch operations,
with ``own`` true the library's call.  ``exact()`` is the operator's definition in 64 bits and
``work()`` the bytes and operations that it cannot do without.
"""
from __future__ import annotations

import math

import torch

own = False

EPS = 1e-5


def listed():
    return [
        # one token at the R1 hidden size: what a decode step pays for a norm (latency)
        dict(name="norm_one_token", op="norm", dtype="bf16", T=1, H=7168),
        # the norm's backward at a 16384-token step of the R1 hidden size
        dict(name="norm_backward_16k", op="norm_backward", dtype="bf16", T=16384, H=7168),
        # both directions of a full-precision norm, no size a multiple of anything
        dict(name="norm_both_f32_odd", op="norm_both", dtype="f32", T=4099, H=1001),
        # the weighted return's gradient at 8192 tokens, top-8 of 256, bf16 residual stream
        dict(name="combine_backward_8k", op="combine_backward", dtype="bf16", dy="bf16", T=8192,
             k=8, E=256, H=7168),
        # the same in f32 for a handful of tokens, odd row length
        dict(name="combine_backward_f32_odd", op="combine_backward", dtype="f32", dy="f32", T=37,
             k=3, E=11, H=1001),
        # the sort's gradient for a 16384-token step, top-8 of 256
        dict(name="permute_backward_16k", op="permute_backward", dtype="bf16", T=16384, k=8, E=256,
             H=7168),
        # the same in f32 for a ragged batch, odd row length
        dict(name="permute_backward_f32_odd", op="permute_backward", dtype="f32", T=997, k=6, E=64,
             H=1333),
        # the router's gradient for a 16384-token step over 256 experts, and for a 64-token one
        dict(name="route_backward_16k", op="route_backward", T=16384, k=8, E=256),
        dict(name="route_backward_64", op="route_backward", T=64, k=8, E=256),
        # the tiny f32 layer's experts at a training batch
        dict(name="experts_backward_f32", op="experts_backward", dtype="f32", T=512, k=2, E=8, H=256,
             I=512, skew=0.3),
        # many experts, skewed routing: hot experts of several tiles, others with a few rows or none
        dict(name="experts_backward_skew", op="experts_backward", dtype="bf16", T=4096, k=6, E=64,
             H=2048, I=1408, skew=1.0),
        # one rank's 32 experts of the R1 shape at a long step: 2048 rows per expert
        dict(name="experts_backward_r1_share", op="experts_backward", dtype="bf16", T=8192, k=8, E=32,
             H=7168, I=2048, skew=0.3),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["norm", "norm_backward", "norm_both", "combine_backward", "permute_backward",
                     "route_backward", "experts_backward", "experts_backward"])
    dtype = rng.choice(["bf16", "bf16", "f32"])
    if op.startswith("norm"):
        H = _log(rng, 64, 12288)
        return dict(op=op, dtype=dtype, T=_log(rng, 1, min(16384, 60_000_000 // H)), H=H)
    E = _log(rng, 4, 256)
    k = rng.randint(2, min(8, E))
    if op == "route_backward":
        return dict(op=op, T=_log(rng, 1, 16384), k=k, E=E)
    if op == "experts_backward":
        E = _log(rng, 2, 48)
        k = rng.randint(1, min(8, E))
        unit = 8 if dtype == "bf16" else 1
        H, I = (unit * _log(rng, 64 // unit, (4096 if unit == 8 else 1024) // unit) for _ in range(2))
        return dict(op=op, dtype=dtype, T=_log(rng, 1, 4096 if unit == 8 else 1024), k=k, E=E, H=H,
                    I=I, skew=round(rng.uniform(0.0, 1.2), 2))
    H = _log(rng, 64, 8192)
    T = _log(rng, 1, min(16384, 400_000_000 // (k * H)))
    c = dict(op=op, dtype=dtype, T=T, k=k, E=E, H=H)
    if op == "combine_backward":
        c["dy"] = rng.choice(["bf16", "f32"])
    return c


def _dtype(name):
    return torch.float32 if name == "f32" else torch.bfloat16


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed) * 7919 + 17)
    op, T = case["op"], case["T"]
    f32 = dict(dtype=torch.float32, device="cuda")

    def normal(*shape, dtype="f32", scale=1.0):
        t = torch.randn(*shape, generator=g, **f32)
        return t.mul_(scale).to(_dtype(dtype))

    s = dict(case)
    if op.startswith("norm"):
        H, dt = case["H"], case["dtype"]
        # rows of a residual stream: their own scale and a small offset each
        x = normal(T, H) * (0.5 + torch.rand(T, 1, generator=g, **f32)) + 0.3 * normal(T, 1)
        s["x"] = x.to(_dtype(dt))
        s["gamma"] = 1.0 + 0.2 * normal(H)
        s["beta"] = 0.1 * normal(H)
        if op != "norm":
            s["dy"] = normal(T, H, dtype=dt, scale=0.05)
            s["dx"] = torch.empty_like(s["x"])
            s["dgamma"], s["dbeta"] = torch.empty(H, **f32), torch.empty(H, **f32)
        if op == "norm_backward":  # what the forward pass left
            xf = s["x"].float()
            s["mean"] = xf.mean(-1)
            s["rstd"] = ((xf - s["mean"][:, None]).square().mean(-1) + EPS).rsqrt()
        else:
            s["y"] = torch.empty_like(s["x"])
            s["mean"], s["rstd"] = torch.empty(T, **f32), torch.empty(T, **f32)
        return s

    k, E = case["k"], case["E"]
    R = T * k
    if op == "experts_backward":
        H, I, dt = case["H"], case["I"], case["dtype"]
        p = torch.softmax(case["skew"] * normal(E), 0)
        ids = torch.multinomial(p, R, replacement=True, generator=g)
        counts = torch.bincount(ids, minlength=E)
        s["offsets"] = torch.zeros(E + 1, dtype=torch.int32, device="cuda")
        s["offsets"][1:] = counts.cumsum(0)
        s["cap"] = int(counts.max())  # the longest expert's rows: what a padded program sizes by
        s["x_perm"] = normal(R, H, dtype=dt)
        s["dy_perm"] = normal(R, H, dtype=dt, scale=0.1)
        w = torch.empty(E, 3 * H * I, dtype=_dtype(dt), device="cuda")
        for e in range(E):
            w[e, :2 * H * I] = normal(2 * H * I, dtype=dt, scale=H ** -0.5)
            w[e, 2 * H * I:] = normal(H * I, dtype=dt, scale=I ** -0.5)
        s["w"] = w
        s["slot_of"] = torch.arange(E, dtype=torch.int32, device="cuda")
        s["dx_perm"] = torch.empty_like(s["x_perm"])
        s["dw"] = torch.empty_like(w)
        return s

    idx = torch.rand(T, E, generator=g, **f32).topk(k, dim=-1).indices
    s["topk_idx"] = idx.to(torch.int32)
    s["topk_w"] = torch.softmax(normal(T, k), -1)
    if op == "route_backward":
        s["dtopk_w"] = normal(T, k, scale=0.5)
        s["dlogits"] = torch.empty(T, E, **f32)
        return s
    src_of = torch.sort(idx.reshape(-1), stable=True).indices
    s["row_of"] = torch.empty(R, dtype=torch.int32, device="cuda")
    s["row_of"][src_of] = torch.arange(R, dtype=torch.int32, device="cuda")
    H, dt = case["H"], case["dtype"]
    if op == "combine_backward":
        s["dy_out"] = normal(T, H, dtype=case["dy"], scale=0.1)
        s["y_perm"] = normal(R, H, scale=0.3)
        s["dy_perm"] = torch.empty(R, H, dtype=_dtype(dt), device="cuda")
        s["dtopk_w"] = torch.empty(T, k, **f32)
    else:
        s["dx_perm"] = normal(R, H, dtype=dt, scale=0.1)
        s["dx"] = torch.empty(T, H, dtype=_dtype(dt), device="cuda")
    return s


# ----------------------------------------------------------------------------
# plain forms
# ----------------------------------------------------------------------------

def _plain_norm(s):
    x = s["x"].float()
    mean = x.mean(-1)
    c = x - mean[:, None]
    rstd = (c.square().mean(-1) + EPS).rsqrt()
    y = c * rstd[:, None] * s["gamma"] + s["beta"]
    return dict(y=y.to(s["x"].dtype), mean=mean, rstd=rstd)


def _plain_norm_backward(s, mean, rstd):
    dy = s["dy"].float()
    xh = (s["x"].float() - mean[:, None]) * rstd[:, None]
    a = dy * s["gamma"]
    dx = rstd[:, None] * (a - a.mean(-1, keepdim=True) - xh * (a * xh).mean(-1, keepdim=True))
    return dict(dx=dx.to(s["x"].dtype), dgamma=(dy * xh).sum(0), dbeta=dy.sum(0))


def _plain_combine_backward(s):
    T, k, H = s["T"], s["k"], s["H"]
    rows = s["row_of"].long()
    dy = s["dy_out"].float()[:, None, :]
    dtopk_w = (s["y_perm"][rows].view(T, k, H) * dy).sum(-1)
    dy_perm = torch.empty(T * k, H, dtype=_dtype(s["dtype"]), device=dy.device)
    dy_perm[rows] = (s["topk_w"][:, :, None] * dy).to(dy_perm.dtype).view(T * k, H)
    return dict(dy_perm=dy_perm, dtopk_w=dtopk_w)


def _plain_permute_backward(s):
    rows = s["row_of"].long()
    dx = s["dx_perm"][rows].float().view(s["T"], s["k"], s["H"]).sum(1)
    return dict(dx=dx.to(s["dx_perm"].dtype))


def _plain_route_backward(s):
    w, dw = s["topk_w"], s["dtopk_w"]
    dl = torch.zeros(s["T"], s["E"], dtype=torch.float32, device=w.device)
    dl.scatter_(1, s["topk_idx"].long(), w * (dw - (w * dw).sum(-1, keepdim=True)))
    return dict(dlogits=dl)


def _plain_experts_backward(s):
    # every expert's rows padded to the longest expert's, then batched products over the experts
    E, H, I, cap = s["E"], s["H"], s["I"], s["cap"]
    off = s["offsets"].long()
    at = torch.arange(cap, device=off.device)
    live = at[None, :] < (off[1:] - off[:-1])[:, None]
    rows = torch.where(live, off[:-1, None] + at[None, :], 0)
    keep = live[:, :, None].float()
    x = s["x_perm"][rows].float() * keep
    dy = s["dy_perm"][rows].float() * keep
    w = s["w"].float()
    wg, wu = w[:, :H * I].view(E, I, H), w[:, H * I:2 * H * I].view(E, I, H)
    wd = w[:, 2 * H * I:].view(E, H, I)
    gate = torch.bmm(x, wg.transpose(1, 2))
    up = torch.bmm(x, wu.transpose(1, 2))
    sig = 1.0 / (1.0 + torch.exp(-gate))
    dh = torch.bmm(dy, wd)
    silu = gate * sig
    dup = dh * silu
    dgate = dh * up * (sig * (1.0 + gate * (1.0 - sig)))
    dx = torch.bmm(dgate, wg) + torch.bmm(dup, wu)
    dt = s["x_perm"].dtype
    dw = torch.cat([torch.bmm(dgate.transpose(1, 2), x).view(E, -1),
                    torch.bmm(dup.transpose(1, 2), x).view(E, -1),
                    torch.bmm(dy.transpose(1, 2), silu * up).view(E, -1)], 1).to(dt)
    return dict(dx_perm=dx[live].to(dt), dw=dw)


# ----------------------------------------------------------------------------
# the library's calls
# ----------------------------------------------------------------------------

def _code(B, name):
    return B.MOE_F32 if name == "f32" else B.MOE_BF16


def _scratch(s, bytes_):
    """The workspace a program keeps from step to step."""
    if "ws" not in s:
        s["ws"] = torch.empty(max(1, bytes_), dtype=torch.uint8, device="cuda")
    return s["ws"]


def _run_own(s):
    from grouped_gemm_weights_amd import binding as B
    op, T = s["op"], s["T"]
    stream = torch.cuda.current_stream()
    if op.startswith("norm"):
        H, dt, out = s["H"], _code(B, s["dtype"]), {}
        if op != "norm_backward":
            B.moe_layer_norm(s["x"], s["gamma"], s["beta"], T, H, EPS, dt, s["y"], s["mean"], s["rstd"],
                             stream)
            out.update(y=s["y"], mean=s["mean"], rstd=s["rstd"])
        if op != "norm":
            need = B.moe_layer_norm_backward_workspace_size(T, H)
            B.moe_layer_norm_backward(s["dy"], s["x"], s["gamma"], s["mean"], s["rstd"], T, H, dt,
                                      s["dx"], s["dgamma"], s["dbeta"], _scratch(s, need), need, stream)
            out.update(dx=s["dx"], dgamma=s["dgamma"], dbeta=s["dbeta"])
        return out
    k, E = s["k"], s["E"]
    if op == "route_backward":
        B.moe_route_backward(s["topk_idx"], s["topk_w"], s["dtopk_w"], T, E, k, s["dlogits"], None, stream)
        return dict(dlogits=s["dlogits"])
    H, dt = s["H"], _code(B, s["dtype"])
    if op == "combine_backward":
        B.moe_combine_backward(s["dy_out"], _code(B, s["dy"]), s["y_perm"], s["row_of"], s["topk_w"], T, k,
                               H, dt, s["dy_perm"], s["dtopk_w"], stream)
        return dict(dy_perm=s["dy_perm"], dtopk_w=s["dtopk_w"])
    if op == "permute_backward":
        B.moe_permute_backward(s["dx_perm"], s["row_of"], T, k, H, dt, s["dx"], stream)
        return dict(dx=s["dx"])
    R, I = T * k, s["I"]
    w = B.wbuf(s["w"], s["w"].shape[1] * s["w"].element_size(), E, E, s["slot_of"])
    need = B.moe_grouped_swiglu_backward_workspace_size(R, E, H, I, dt)
    B.moe_grouped_swiglu_backward(s["x_perm"], s["dy_perm"], s["offsets"], R, E, H, I, dt, w,
                                  _scratch(s, need), need, s["dx_perm"], s["dw"], None, stream)
    return dict(dx_perm=s["dx_perm"], dw=s["dw"])


def run(state):
    if own:
        return _run_own(state)
    op = state["op"]
    if op == "norm":
        return _plain_norm(state)
    if op == "norm_backward":
        return _plain_norm_backward(state, state["mean"], state["rstd"])
    if op == "norm_both":
        out = _plain_norm(state)
        out.update(_plain_norm_backward(state, out["mean"], out["rstd"]))
        return out
    return dict(combine_backward=_plain_combine_backward, permute_backward=_plain_permute_backward,
                route_backward=_plain_route_backward,
                experts_backward=_plain_experts_backward)[op](state)


# ----------------------------------------------------------------------------
# cost and definition
# ----------------------------------------------------------------------------

def _size(name):
    return 4 if name == "f32" else 2


def work(case):
    op, T = case["op"], case["T"]
    if op.startswith("norm"):
        n, H, e = T * case["H"], case["H"], _size(case["dtype"])
        forward, backward = 2 * n * e + 8 * H + 8 * T, 3 * n * e + 12 * H + 8 * T
        return dict(norm=dict(bytes=forward, flops=8 * n), norm_backward=dict(bytes=backward, flops=14 * n),
                    # x is read once for both directions, gamma and the statistics too
                    norm_both=dict(bytes=4 * n * e + 16 * H + 8 * T, flops=22 * n))[op]
    R, E = T * case["k"], case["E"]
    if op == "route_backward":
        return dict(bytes=12 * R + 4 * T * E, flops=4 * R)
    H, e = case["H"], _size(case["dtype"])
    if op == "combine_backward":
        return dict(bytes=T * H * _size(case["dy"]) + R * H * (4 + e) + 12 * R, flops=3 * R * H)
    if op == "permute_backward":
        return dict(bytes=(R + T) * H * e + 4 * R, flops=R * H)
    # rows in and out, every expert's weights in and their gradient out; g and u are recomputed
    return dict(bytes=3 * R * H * e + 6 * E * H * case["I"] * e, flops=16 * R * H * case["I"])


def exact(case, seed):
    s = prepare(case, seed)
    d = {n: t.double() for n, t in s.items() if torch.is_tensor(t) and t.is_floating_point() and n != "w"}
    op, T = case["op"], case["T"]
    if op.startswith("norm"):
        H = case["H"]
        out = {}
        x, mu, r = d["x"], d["mean"], d["rstd"]
        if op != "norm_backward":
            mu = x.sum(1) / H
            r = 1.0 / torch.sqrt(((x * x).sum(1) / H - mu * mu) + EPS)
            y = torch.addcmul(d["beta"], (x - mu.unsqueeze(1)) * d["gamma"], r.unsqueeze(1))
            out.update(y=y, mean=mu, rstd=r)
        if op != "norm":
            # the Jacobian of a row is r (1 - (11' + xh xh') / H), applied to dy * gamma
            xh = (x - mu.unsqueeze(1)).mul_(r.unsqueeze(1))
            v = d["dy"] * d["gamma"]
            along_one, along_x = v.sum(1) / H, torch.linalg.vecdot(v, xh) / H
            dx = (v - along_one.unsqueeze(1) - along_x.unsqueeze(1) * xh) * r.unsqueeze(1)
            ones = torch.ones(1, T, dtype=torch.float64, device=x.device)
            out.update(dx=dx, dgamma=(ones @ (d["dy"] * xh))[0], dbeta=(ones @ d["dy"])[0])
        return out
    k, E = case["k"], case["E"]
    if op == "route_backward":
        # the softmax's Jacobian diag(w) - w w', slot by slot
        w, idx = d["topk_w"], s["topk_idx"].long()
        dl = torch.zeros(T, E, dtype=torch.float64, device=w.device)
        t = torch.arange(T, device=w.device)
        for j in range(k):
            for i in range(k):
                dl[t, idx[:, j]] += w[:, j] * ((1.0 if i == j else 0.0) - w[:, i]) * d["dtopk_w"][:, i]
        return dict(dlogits=dl)
    H = case["H"]
    if op == "combine_backward":
        r = s["row_of"].long().view(T, k)
        dy_perm = torch.empty(T * k, H, dtype=torch.float64, device=r.device)
        dtopk_w = torch.empty(T, k, dtype=torch.float64, device=r.device)
        for j in range(k):
            dy_perm[r[:, j]] = d["topk_w"][:, j:j + 1] * d["dy_out"]
            dtopk_w[:, j] = torch.linalg.vecdot(d["dy_out"], d["y_perm"][r[:, j]])
        return dict(dy_perm=dy_perm, dtopk_w=dtopk_w)
    if op == "permute_backward":
        r = s["row_of"].long().view(T, k)
        dx = torch.zeros(T, H, dtype=torch.float64, device=r.device)
        for j in range(k):
            dx += d["dx_perm"][r[:, j]]
        return dict(dx=dx)
    I = case["I"]
    if 16.0 * T * k * H * I > 2e13:
        return None
    off = s["offsets"].tolist()
    dx_perm = torch.zeros_like(d["x_perm"])
    dw = torch.zeros(E, 3 * H * I, dtype=torch.float64, device=dx_perm.device)
    for e in range(E):
        a, b = off[e], off[e + 1]
        if a == b:
            continue
        x, dy = d["x_perm"][a:b], d["dy_perm"][a:b]
        w = s["w"][e].double()
        wgu, wd = w[:2 * H * I].view(2 * I, H), w[2 * H * I:].view(H, I)
        gate, up = (x @ wgu.t()).split(I, 1)
        sg = torch.sigmoid(gate)
        dh = dy @ wd
        dgu = torch.cat([dh * up * (sg + gate * sg * (1 - sg)), dh * gate * sg], 1)
        dx_perm[a:b] = dgu @ wgu
        dw[e, :2 * H * I] = (dgu.t() @ x).reshape(-1)
        dw[e, 2 * H * I:] = (dy.t() @ (gate * sg * up)).reshape(-1)
    return dict(dx_perm=dx_perm, dw=dw)
