"""The 8-bit pass of the MoE block and its neighbours, operator by operator: what is run, on what, and
what it costs.

The operators are the root-mean-square norm with the residual's addition (``moe_rms_norm`` and its
backward), the quantisation to 8 bits with block scales (``moe_mx_quantize``), the products grouped
by expert (``moe_grouped_gemm``, its backward, and ``moe_grouped_gemm_mx`` on 8-bit operands) and the
dropout in front of the residual (``moe_dropout_add`` and its backward).

8-bit rows are e4m3 values with one power-of-two scale for each 32 of them (a byte, the exponent
plus 127); a row's scales are padded with zero bytes to a multiple of 16.

``listed()`` and ``draw()`` give cases, ``prepare()`` the inputs a program has in hand, ``run()``
one pass through the operator: with ``own`` false its plain form in elementary torch operations,
with ``own`` true the library's call.  ``exact()`` is the operator's definition in 64 bits and
``work()`` the bytes and operations that it cannot do without.
"""
from __future__ import annotations

import math

import torch

own = False

EPS = 1e-6
BLOCK = 32  # values that share a scale


def listed():
    return [
        # a decode step of 64 tokens at the R1 hidden size: the stream's new sum, its norm for the
        # router and the same in 8 bits for the experts (latency)
        dict(name="norm_mx_decode", op="norm", dtype="bf16", T=64, H=7168, residual=True, mx=True,
             backward=False),
        # the same for a 16384-token prompt
        dict(name="norm_mx_16k", op="norm", dtype="bf16", T=16384, H=7168, residual=True, mx=True,
             backward=False),
        # a full-precision training step of the norm, no size a multiple of anything
        dict(name="norm_train_f32_odd", op="norm", dtype="f32", T=4099, H=1001, residual=True, mx=False,
             backward=True),
        # a checkpoint's weights to 8 bits as they are loaded: gate and up rows of one R1 expert
        dict(name="quantize_weights", op="quantize", dtype="bf16", rows=4096, cols=7168, swiglu=False),
        # the experts' activation between their two products, 8192 tokens top-8, to 8 bits
        dict(name="quantize_swiglu_64k", op="quantize", dtype="bf16", rows=65536, cols=2048, swiglu=True),
        # 8-bit decode: 64 tokens top-8 over one rank's 64 experts, gate and up in one product
        dict(name="product_mx_decode", op="product", dtype="mx", out="bf16", T=64, k=8, E=64, K=7168,
             N=4096, skew=0.5, gather=True, backward=False),
        # 8-bit prompt: 8192 tokens top-8 over 32 experts, 2048 rows an expert
        dict(name="product_mx_r1_share", op="product", dtype="mx", out="bf16", T=8192, k=8, E=32, K=7168,
             N=4096, skew=0.3, gather=True, backward=False),
        # bf16 experts of another shape, skewed routing: hot experts beside nearly empty ones
        dict(name="product_bf16_skew", op="product", dtype="bf16", out="f32", T=2048, k=6, E=64, K=2048,
             N=1408, skew=1.0, gather=True, backward=False),
        # the same experts' training step: output, input and weight gradients
        dict(name="product_train_bf16", op="product", dtype="bf16", out="bf16", T=4096, k=6, E=64, K=1408,
             N=2048, skew=1.0, gather=False, backward=True),
        # a small full-precision layer's training step, odd sizes
        dict(name="product_train_f32_odd", op="product", dtype="f32", out="f32", T=257, k=3, E=11, K=331,
             N=517, skew=0.5, gather=False, backward=True),
        # dropout of the block's fp32 output in front of the residual, a small training batch (latency)
        dict(name="dropout_small", op="dropout", x="f32", dtype="bf16", T=61, H=1000, p=0.1, residual=True,
             backward=False),
        # both directions over a 16384-token step of the R1 hidden size
        dict(name="dropout_train_16k", op="dropout", x="f32", dtype="bf16", T=16384, H=7168, p=0.1,
             residual=True, backward=True),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["norm", "norm", "quantize", "product", "product", "product", "dropout"])
    dtype = rng.choice(["bf16", "bf16", "f32"])
    if op == "norm":
        mx = rng.random() < 0.5
        H = BLOCK * _log(rng, 2, 384) if mx else _log(rng, 64, 12288)
        return dict(op=op, dtype=dtype, T=_log(rng, 1, min(16384, 40_000_000 // H)), H=H,
                    residual=rng.random() < 0.7, mx=mx, backward=not mx and rng.random() < 0.7)
    if op == "quantize":
        cols = BLOCK * _log(rng, 1, 256)
        return dict(op=op, dtype=dtype, rows=_log(rng, 1, min(65536, 60_000_000 // cols)), cols=cols,
                    swiglu=rng.random() < 0.5)
    if op == "dropout":
        H = _log(rng, 64, 8192)
        return dict(op=op, x=rng.choice(["f32", "bf16"]), dtype=dtype, T=_log(rng, 1, min(16384, 60_000_000 // H)),
                    H=H, p=rng.choice([0.0, 0.05, 0.1, 0.3, 0.5]), residual=rng.random() < 0.7,
                    backward=rng.random() < 0.5)
    dtype = rng.choice(["mx", "mx", "bf16", "bf16", "f32"])
    E = _log(rng, 1, 64)
    k = rng.randint(1, min(8, E))
    unit = dict(mx=32, bf16=8, f32=1)[dtype]
    top = 1024 if dtype == "f32" else 4096
    K = unit * _log(rng, max(1, 64 // unit), top // unit)
    unit = dict(mx=8, bf16=8, f32=1)[dtype]
    N = unit * _log(rng, max(1, 64 // unit), top // unit)
    backward = dtype != "mx" and rng.random() < 0.5
    return dict(op=op, dtype=dtype, out="f32" if dtype == "f32" else rng.choice(["bf16", "f32"]),
                T=_log(rng, 1, 1024 if dtype == "f32" else 4096), k=k, E=E, K=K, N=N,
                skew=round(rng.uniform(0.0, 1.2), 2), gather=not backward and rng.random() < 0.5,
                backward=backward)


def _dtype(name):
    return torch.float32 if name == "f32" else torch.bfloat16


def _pitch(cols):
    """Bytes of a row's scales: one for each block, padded to a multiple of 16."""
    return 16 * -(-cols // (16 * BLOCK))


def _power(e, dtype=torch.float32):
    """2^e for whole e from -149 to 127, exactly."""
    return ((e.long() + 1023) << 52).view(torch.float64).to(dtype)


def _to_8_bits(y):
    """e4m3 values and scale bytes of the rows of y (fp32).  The scale is the smallest power of two
    that leaves no value of its block above 448, the largest of e4m3 (1.75 * 2^8)."""
    rows, cols = y.shape
    b = y.view(rows, cols // BLOCK, BLOCK)
    bits = b.abs().amax(-1).view(torch.int32)
    byte = ((bits >> 23) - 8 + ((bits & 0x7FFFFF) > 0x600000).int()).clamp(0, 254)
    q = (b * _power(127 - byte)[:, :, None]).to(torch.float8_e4m3fn)
    scales = torch.zeros(rows, _pitch(cols), dtype=torch.uint8, device=y.device)
    scales[:, :cols // BLOCK] = byte.to(torch.uint8)
    return q.view(rows, cols), scales


def _from_8_bits(q, scales, dtype=torch.float32):
    """The values that e4m3 bytes and their scale bytes stand for: [..., cols] and [..., pitch]."""
    cols = q.shape[-1]
    e = scales[..., :cols // BLOCK].to(torch.int32) - 127
    v = q.view(torch.float8_e4m3fn).to(dtype).view(*q.shape[:-1], cols // BLOCK, BLOCK)
    return (v * _power(e, dtype)[..., None]).view(q.shape)


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed) * 7919 + 23)
    f32 = dict(dtype=torch.float32, device="cuda")

    def normal(*shape, dtype="f32", scale=1.0):
        return torch.randn(*shape, generator=g, **f32).mul_(scale).to(_dtype(dtype))

    def empty(*shape, dtype="f32"):
        return torch.empty(*shape, dtype=_dtype(dtype), device="cuda")

    def empty_8(rows, cols):
        return (torch.empty(rows, cols, dtype=torch.uint8, device="cuda"),
                torch.empty(rows, _pitch(cols), dtype=torch.uint8, device="cuda"))

    s = dict(case)
    op = case["op"]
    if op == "norm":
        T, H, dt = case["T"], case["H"], case["dtype"]
        # the residual stream, rows of their own scale, and what a block adds to it
        s["x"] = (normal(T, H) * (0.5 + torch.rand(T, 1, generator=g, **f32))).to(_dtype(dt))
        s["gamma"] = 1.0 + 0.2 * normal(H)
        s["y"], s["rstd"] = empty(T, H, dtype=dt), empty(T)
        if case["residual"]:
            s["res"] = normal(T, H, dtype=dt, scale=0.7)
            s["sum"] = empty(T, H, dtype=dt)
        if case["mx"]:
            s["q"], s["scales"] = empty_8(T, H)
        if case["backward"]:
            s["dy"], s["dsum"] = normal(T, H, dtype=dt, scale=0.05), normal(T, H, dtype=dt, scale=0.05)
            s["dx"], s["dgamma"] = empty(T, H, dtype=dt), empty(H)
    elif op == "quantize":
        rows, cols, dt = case["rows"], case["cols"], case["dtype"]
        if case["swiglu"]:  # gate and up of each row, side by side
            s["src"] = normal(rows, 2 * cols, dtype=dt)
        else:  # a weight matrix
            s["src"] = normal(rows, cols, dtype=dt, scale=cols ** -0.5)
        s["q"], s["scales"] = empty_8(rows, cols)
    elif op == "dropout":
        n = (case["T"], case["H"])
        s["src"] = normal(*n, dtype=case["x"])
        s["res"] = normal(*n, dtype=case["dtype"]) if case["residual"] else None
        # the generator's key and the step's number, as a program keeps them on the GPU
        s["rng"] = torch.tensor([int(seed) * 1_000_003 + 12_345_678_901, int(seed) + 3], dtype=torch.int64,
                                device="cuda")
        s["y"] = empty(*n, dtype=case["dtype"])
        if case["backward"]:
            s["dy"] = normal(*n, dtype=case["dtype"], scale=0.05)
            s["dx"] = empty(*n, dtype=case["x"])
    else:
        T, k, E, K, N, dt = (case[n] for n in ("T", "k", "E", "K", "N", "dtype"))
        R = T * k
        p = torch.softmax(case["skew"] * normal(E), 0)
        ids = torch.multinomial(p.expand(T, E).contiguous(), k, generator=g)
        counts = torch.bincount(ids.view(-1), minlength=E)
        s["offsets"] = torch.zeros(E + 1, dtype=torch.int32, device="cuda")
        s["offsets"][1:] = counts.cumsum(0)
        s["cap"] = int(counts.max())  # the longest expert's rows: what a padded program sizes by
        s["src_of"] = torch.sort(ids.view(-1), stable=True).indices.int() if case["gather"] else None
        x = normal(T if case["gather"] else R, K, dtype="f32" if dt == "mx" else dt)
        if dt == "mx":
            q, s["xs"] = _to_8_bits(x)
            s["x"] = q.view(torch.uint8)
            # an expert's block: its matrix, then the matrix's scales
            s["w"] = torch.empty(E, N * (K + _pitch(K)), dtype=torch.uint8, device="cuda")
            for e in range(E):
                q, ws = _to_8_bits(normal(N, K, scale=K ** -0.5))
                s["w"][e, :N * K] = q.view(torch.uint8).view(-1)
                s["w"][e, N * K:] = ws.view(-1)
        else:
            s["x"] = x
            s["w"] = torch.empty(E, N * K, dtype=_dtype(dt), device="cuda")
            for e in range(E):
                s["w"][e] = normal(N * K, dtype=dt, scale=K ** -0.5)
        s["slot_of"] = torch.arange(E, dtype=torch.int32, device="cuda")
        s["y"] = empty(R, N, dtype=case["out"])
        if case["backward"]:
            s["dy"] = normal(R, N, dtype=dt, scale=0.1)
            s["dx"] = torch.empty_like(s["x"])
            s["dw"] = torch.empty_like(s["w"])
    return s


# ----------------------------------------------------------------------------
# plain forms
# ----------------------------------------------------------------------------

def _values(q, scales):
    """8-bit outputs as the values they stand for, element and scale apart."""
    return dict(q=q.view(torch.float8_e4m3fn), scales=scales.view(torch.float8_e8m0fnu))


def _plain_norm(s):
    dt, out = s["x"].dtype, {}
    stream = s["x"]
    if s["residual"]:  # the norm is that of the sum as it is stored
        stream = (s["x"].float() + s["res"].float()).to(dt)
        out["sum"] = stream
    v = stream.float()
    rstd = (v.square().mean(-1) + EPS).rsqrt()
    y = v * rstd[:, None] * s["gamma"]
    out.update(y=y.to(dt), rstd=rstd)
    if s["mx"]:
        out.update(_values(*_to_8_bits(y)))
    if s["backward"]:
        xh = v * rstd[:, None]
        a = s["dy"].float() * s["gamma"]
        dx = rstd[:, None] * (a - xh * (a * xh).mean(-1, keepdim=True)) + s["dsum"].float()
        out.update(dx=dx.to(dt), dgamma=(s["dy"].float() * xh).sum(0))
    return out


def _plain_quantize(s):
    v = s["src"].float()
    if s["swiglu"]:
        gate, up = v[:, :s["cols"]], v[:, s["cols"]:]
        v = gate / (1.0 + torch.exp(-gate)) * up
    return _values(*_to_8_bits(v))


def _plain_keep(s):
    """Philox4x32-10: counter (element / 4, step), key the seed, four 32-bit words a counter.  An
    element is kept where its word is not below p 2^32."""
    n, mask = s["T"] * s["H"], 0xFFFFFFFF
    seed, step = s["rng"][0], s["rng"][1]
    at = torch.arange(-(-n // 4), device="cuda")
    c = [at & mask, at >> 32, step & mask, (step >> 32) & mask]
    key = [seed & mask, (seed >> 32) & mask]
    for _ in range(10):
        a, b = c[0] * 0xD2511F53, c[2] * 0xCD9E8D57  # 64-bit products, of which all bits are kept
        c = [((b >> 32) & mask) ^ c[1] ^ key[0], b & mask, ((a >> 32) & mask) ^ c[3] ^ key[1], a & mask]
        key = [(key[0] + 0x9E3779B9) & mask, (key[1] + 0xBB67AE85) & mask]
    words = torch.stack([w.expand(at.shape) for w in c], 1).view(-1)[:n]
    return (words >= int(s["p"] * 2.0 ** 32)).view(s["T"], s["H"])


def _plain_dropout(s):
    keep, scale = _plain_keep(s), 1.0 / (1.0 - s["p"])
    y = torch.where(keep, s["src"].float() * scale, 0.0)
    if s["residual"]:
        y = y + s["res"].float()
    out = dict(y=y.to(_dtype(s["dtype"])))
    if s["backward"]:
        out["dx"] = torch.where(keep, s["dy"].float() * scale, 0.0).to(_dtype(s["x"]))
    return out


def _plain_product(s):
    # every expert's rows padded to the longest expert's, then batched products over the experts
    E, K, N, cap = s["E"], s["K"], s["N"], s["cap"]
    off = s["offsets"].long()
    at = torch.arange(cap, device=off.device)
    live = at[None, :] < (off[1:] - off[:-1])[:, None]
    rows = torch.where(live, off[:-1, None] + at[None, :], 0)
    keep = live[:, :, None].float()
    from_row = s["src_of"].long()[rows] // s["k"] if s["gather"] else rows
    if s["dtype"] == "mx":
        x = _from_8_bits(s["x"], s["xs"])[from_row]
        w = _from_8_bits(s["w"][:, :N * K].view(E, N, K),
                         s["w"][:, N * K:].view(E, N, _pitch(K)))
    else:
        x, w = s["x"][from_row].float(), s["w"].float().view(E, N, K)
    x = x * keep
    out = dict(y=torch.bmm(x, w.transpose(1, 2))[live].to(_dtype(s["out"])))
    if s["backward"]:
        dy = s["dy"][rows].float() * keep
        out.update(dx=torch.bmm(dy, w)[live].to(s["x"].dtype),
                   dw=torch.bmm(dy.transpose(1, 2), x).to(s["x"].dtype).view(E, -1))
    return out


# ----------------------------------------------------------------------------
# the library's calls
# ----------------------------------------------------------------------------

def _code(B, name):
    return B.MOE_F32 if name == "f32" else B.MOE_BF16


def _run_own(s):
    from grouped_gemm_weights_amd import binding as B
    stream = torch.cuda.current_stream()
    op, out = s["op"], {}
    if op == "norm":
        T, H, dt = s["T"], s["H"], _code(B, s["dtype"])
        B.moe_rms_norm(s["x"], s.get("res"), s["gamma"], T, H, EPS, dt, s.get("sum"), s["y"], s.get("q"),
                       s.get("scales"), s["rstd"], stream)
        out.update(y=s["y"], rstd=s["rstd"])
        if s["residual"]:
            out["sum"] = s["sum"]
        if s["mx"]:
            out.update(_values(s["q"], s["scales"]))
        if s["backward"]:
            need = B.moe_rms_norm_backward_workspace_size(T, H)
            if "ws" not in s:  # a program keeps its workspace from step to step
                s["ws"] = torch.empty(max(1, need), dtype=torch.uint8, device="cuda")
            B.moe_rms_norm_backward(s["dy"], s["dsum"], s["sum"] if s["residual"] else s["x"], s["gamma"],
                                    s["rstd"], T, H, dt, s["dx"], s["dgamma"], s["ws"], need, stream)
            out.update(dx=s["dx"], dgamma=s["dgamma"])
        return out
    if op == "quantize":
        B.moe_mx_quantize(s["src"], s["rows"], s["cols"], _code(B, s["dtype"]), s["swiglu"], s["q"],
                          s["scales"], stream)
        return _values(s["q"], s["scales"])
    if op == "dropout":
        n, xdt, dt = s["T"] * s["H"], _code(B, s["x"]), _code(B, s["dtype"])
        B.moe_dropout_add(s["src"], xdt, s["res"], n, s["p"], s["rng"], dt, s["y"], stream)
        out["y"] = s["y"]
        if s["backward"]:
            B.moe_dropout_add_backward(s["dy"], dt, n, s["p"], s["rng"], xdt, s["dx"], stream)
            out["dx"] = s["dx"]
        return out
    E, K, N, R = s["E"], s["K"], s["N"], s["T"] * s["k"]
    w = B.wbuf(s["w"], s["w"].shape[1] * s["w"].element_size(), E, E, s["slot_of"])
    if s["dtype"] == "mx":
        B.moe_grouped_gemm_mx(s["x"], s["xs"], s["src_of"], s["k"], s["offsets"], R, E, K, N, w, 0, N * K,
                              _code(B, s["out"]), s["y"], None, stream)
        return dict(y=s["y"])
    dt = _code(B, s["dtype"])
    B.moe_grouped_gemm(s["x"], s["src_of"], s["k"], s["offsets"], R, E, K, N, dt, w, 0, _code(B, s["out"]),
                       s["y"], None, stream)
    out["y"] = s["y"]
    if s["backward"]:
        B.moe_grouped_gemm_backward(s["x"], s["dy"], s["offsets"], R, E, K, N, dt, w, 0, s["dx"], s["dw"],
                                    None, stream)
        out.update(dx=s["dx"], dw=s["dw"])
    return out


def run(state):
    if own:
        return _run_own(state)
    return dict(norm=_plain_norm, quantize=_plain_quantize, product=_plain_product,
                dropout=_plain_dropout)[state["op"]](state)


# ----------------------------------------------------------------------------
# cost and definition
# ----------------------------------------------------------------------------

def _size(name):
    return dict(f32=4, bf16=2, mx=1)[name]


def work(case):
    op = case["op"]
    if op == "norm":
        T, H, e = case["T"], case["H"], _size(case["dtype"])
        # x in and y out; the residual in and the sum out; 8-bit rows and scales out
        rows = (4 if case["residual"] else 2) * e * H + ((H + _pitch(H)) if case["mx"] else 0) + 4
        # the stream is read once for both directions; two gradients in and one out
        rows += 3 * e * H if case["backward"] else 0
        return dict(bytes=T * rows + 4 * H * (2 if case["backward"] else 1),
                    flops=T * H * (5 + (12 if case["backward"] else 0) + (4 if case["mx"] else 0)))
    if op == "quantize":
        n, c = case["rows"], case["cols"]
        wide = 2 if case["swiglu"] else 1
        return dict(bytes=n * (c * wide * _size(case["dtype"]) + c + _pitch(c)), flops=n * c * (4 + 5 * wide))
    if op == "dropout":
        n, x, o = case["T"] * case["H"], _size(case["x"]), _size(case["dtype"])
        both = 2 if case["backward"] else 1
        return dict(bytes=n * (x + o + (o if case["residual"] else 0) + (x + o if case["backward"] else 0)) + 16,
                    flops=2 * n * both)
    T, E, K, N = (case[n] for n in ("T", "E", "K", "N"))
    R, e = T * case["k"], _size(case["dtype"])
    rows_in, used = (T if case["gather"] else R), min(E, R)
    scales = _pitch(K) if case["dtype"] == "mx" else 0
    total = rows_in * (K * e + scales) + used * N * (K * e + scales) + R * N * _size(case["out"])
    if case["backward"]:  # dy in, dx and every expert's dw out; x and the weights are in already
        total += R * (N + K) * e + E * N * K * e
    return dict(bytes=total, flops=2 * R * K * N * (3 if case["backward"] else 1))


def _exact_8_bits(v):
    """Elements before they are rounded, over their block's scale, and the scales."""
    rows, cols = v.shape
    b = v.view(rows, -1, BLOCK)
    top = b.abs().max(-1).values
    e = torch.ceil(torch.log2(top / 448.0))
    e = e + (top > 448.0 * torch.exp2(e)).double() - (top <= 448.0 * torch.exp2(e - 1)).double()
    e = e.clamp(-127, 127)
    scales = torch.full((rows, _pitch(cols)), 2.0 ** -127, dtype=torch.float64, device=v.device)
    scales[:, :cols // BLOCK] = torch.exp2(e)
    return dict(q=(b / torch.exp2(e)[:, :, None]).view(rows, cols), scales=scales)


def _exact_keep(s):
    """The generator again, its 64-bit products put together from halves of 16 bits."""
    n, low = s["T"] * s["H"], (1 << 32) - 1
    seed, step = (int(v) for v in s["rng"].tolist())
    i = torch.arange((n + 3) // 4, device="cuda")

    def product(a, b):
        part0, part1 = (b & 0xFFFF) * a, (b >> 16) * a
        high = (part1 + (part0 >> 16)) >> 16
        return high, ((part1 << 16) + part0) & low

    x0, x1 = i & low, i >> 32
    x2, x3 = torch.full_like(i, step & low), torch.full_like(i, (step >> 32) & low)
    k0, k1 = seed & low, (seed >> 32) & low
    for turn in range(10):
        h0, l0 = product(0xD2511F53, x0)
        h2, l2 = product(0xCD9E8D57, x2)
        x0, x1, x2, x3 = h2 ^ x1 ^ k0, l2, h0 ^ x3 ^ k1, l0
        k0, k1 = (k0 + 0x9E3779B9) & low, (k1 + 0xBB67AE85) & low
    u = torch.stack((x0, x1, x2, x3), -1).reshape(-1)[:n].double()
    return (u >= math.floor(s["p"] * 4294967296.0)).view(s["T"], s["H"]).double()


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    d = {n: t.double() for n, t in s.items() if torch.is_tensor(t) and t.is_floating_point() and n != "w"}
    if op == "norm":
        out, v = {}, d["x"]
        if case["residual"]:
            out["sum"] = d["x"] + d["res"]
            v = out["sum"].to(s["x"].dtype).double()  # the norm is that of the stored sum
        H = case["H"]
        r = 1.0 / torch.sqrt(torch.linalg.vecdot(v, v) / H + EPS)
        y = v * d["gamma"] * r.unsqueeze(1)
        out.update(y=y, rstd=r)
        if case["mx"]:
            out.update(_exact_8_bits(y))
        if case["backward"]:
            # the Jacobian of a row is r (1 - xh xh' / H), applied to dy * gamma
            xh = v * r.unsqueeze(1)
            a = d["dy"] * d["gamma"]
            along = torch.linalg.vecdot(a, xh) / H
            out["dx"] = d["dsum"] + (a - along.unsqueeze(1) * xh) * r.unsqueeze(1)
            out["dgamma"] = (torch.ones(1, case["T"], dtype=torch.float64, device=v.device) @ (d["dy"] * xh))[0]
        return out
    if op == "quantize":
        v = d["src"]
        if case["swiglu"]:
            gate, up = v.split(case["cols"], 1)
            v = gate * torch.sigmoid(gate) * up
        return _exact_8_bits(v)
    if op == "dropout":
        m = _exact_keep(s) / (1.0 - case["p"])
        y = d["src"] * m
        out = dict(y=y + d["res"] if case["residual"] else y)
        if case["backward"]:
            out["dx"] = d["dy"] * m
        return out
    T, k, E, K, N = (case[n] for n in ("T", "k", "E", "K", "N"))
    R = T * k
    if 2.0 * R * K * N * (3 if case["backward"] else 1) > 2e13:
        return None
    off = s["offsets"].tolist()
    y = torch.zeros(R, N, dtype=torch.float64, device="cuda")
    out = dict(y=y)
    if case["backward"]:
        out.update(dx=torch.zeros_like(d["x"]), dw=torch.zeros(E, N * K, dtype=torch.float64, device="cuda"))
    for e in range(E):
        a, b = off[e], off[e + 1]
        if a == b:
            continue
        at = torch.arange(a, b, device="cuda") if not case["gather"] else torch.div(
            s["src_of"][a:b].long(), k, rounding_mode="floor")
        if case["dtype"] == "mx":
            block = s["w"][e]
            x = _from_8_bits(s["x"][at], s["xs"][at], torch.float64)
            w = _from_8_bits(block[:N * K].view(N, K), block[N * K:].view(N, -1),
                             torch.float64)
        else:
            x, w = d["x"][at], s["w"][e].double().view(N, K)
        y[a:b] = x @ w.t()
        if case["backward"]:
            out["dx"][a:b] = d["dy"][a:b] @ w
            out["dw"][e] = (d["dy"][a:b].t() @ x).reshape(-1)
    return out
