"""Cases of the dense operators around the quantised FFN, in plain form and as library calls.

* swiglu_linear: the 16-bit gated projection h = silu(x Wg^T) * (x Wu^T), for serving
  (forward) and for training (forward and backward);
* int8_linear: the INT8 matrix product with a scale per token and per output channel;
* block_norm: the norms before and after a block with its gate and residual scale,
  r = res + alpha * gate * N(y; w_post), n = N(r; w_pre), forward and backward;
* int8_block: the last two as used together: residual stream -> norm with INT8 codes ->
  INT8 product -> norm after the block, gate, residual scale.

``own`` selects what ``run`` does: False, elementary torch operations in 32 bits (exact
integer sums for the INT8 product); True, the library's entry points.
"""
import math

import torch

own = False

EPS = 1e-6
DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}


def listed():
    return [
        # one decoded token through the gated projection of a 2048 / 8192 dense FFN
        dict(name="swiglu_t1", kind="swiglu", t=1, h=2048, i=8192, dtype="bf16"),
        # a decode batch through the 16-bit shared expert of a 7168-wide layer
        dict(name="swiglu_t64", kind="swiglu", t=64, h=7168, i=2048, dtype="bf16"),
        # a prefill chunk through the same expert
        dict(name="swiglu_t4096", kind="swiglu", t=4096, h=7168, i=2048, dtype="bf16"),
        # a training step's gated projection on a 4096-token batch of the dense FFN
        dict(name="swiglu_train_t4096", kind="swiglu_train", t=4096, h=2048, i=8192, dtype="bf16"),
        # a short packed batch and widths that no tile divides, in fp16
        dict(name="swiglu_train_ragged", kind="swiglu_train", t=777, h=1000, i=2728, dtype="fp16"),
        # one token through a square linear
        dict(name="int8_t1", kind="int8", t=1, k=2048, n=2048, dtype="bf16", bias=False),
        # a decode batch through the down projection of the dense FFN
        dict(name="int8_t16", kind="int8", t=16, k=8192, n=2048, dtype="bf16", bias=False),
        # prefill through the stacked gate and up projections of the dense FFN
        dict(name="int8_t2048", kind="int8", t=2048, k=2048, n=16384, dtype="bf16", bias=False),
        # odd lengths with a bias and an fp32 result (a classification or output head)
        dict(name="int8_ragged", kind="int8", t=333, k=1040, n=1001, dtype="fp32", bias=True),
        # one token: residual stream -> INT8 codes -> product -> norm, gate, residual
        dict(name="int8_block_t1", kind="int8_block", t=1, h=2048, dtype="bf16"),
        # the norms between two blocks of a 7168-wide model on a prefill chunk
        dict(name="norm_t4096", kind="norm", t=4096, h=7168, gate="channel", dtype="bf16"),
        # the same boundary in a training step, the gate per token (a shared expert's)
        dict(name="norm_train_t4096", kind="norm_train", t=4096, h=2048, gate="token", dtype="bf16"),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _width(rng, lo, hi, step):
    """A width between lo and hi, a multiple of step; one in two a multiple of 128."""
    w = _log_int(rng, lo, hi)
    step = 128 if rng.random() < 0.5 else step
    return max(step, w // step * step)


def draw(rng):
    kind = rng.choice(["swiglu", "swiglu_train", "int8", "int8", "int8_block", "norm", "norm_train"])
    t = _log_int(rng, 1, 4096)
    if kind in ("swiglu", "swiglu_train"):
        t = t if kind == "swiglu" else max(t, _log_int(rng, 1, 4096))
        h = _width(rng, 64, 7168, 8)
        i = _width(rng, 64, 8192, 8)
        while t * h * i > 4096 * 2048 * 8192:
            t = (t + 1) // 2
        return dict(kind=kind, t=t, h=h, i=i, dtype=rng.choice(["bf16", "fp16"]))
    if kind == "int8":
        k = _width(rng, 64, 16384, 16)
        n = _log_int(rng, 16, 16384)
        while t * n * k > 2048 * 2048 * 16384:
            t = (t + 1) // 2
        return dict(kind=kind, t=t, k=k, n=n, dtype=rng.choice(["bf16", "fp16", "fp32"]), bias=rng.random() < 0.5)
    if kind == "int8_block":
        return dict(kind=kind, t=min(t, 2048), h=_width(rng, 64, 7168, 16), dtype=rng.choice(["bf16", "fp16"]))
    gate = rng.choice(["none", "channel", "token", "element"])
    dtype = rng.choice(["bf16", "fp16", "fp32"])
    h = _width(rng, 64, 7168, 1)
    return dict(kind=kind, t=t, h=h, gate=gate, dtype=dtype)


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(int(seed))
    dt = DTYPES[case["dtype"]]

    def normal(*shape, std=1.0):
        return torch.randn(*shape, generator=gen, device="cuda") * std

    def tokens(t, w):
        # unit tokens with 1 % of the channels ten times larger, as hidden states have them
        x = normal(t, w)
        big = torch.rand(w, generator=gen, device="cuda") < 0.01
        return torch.where(big, x * 10, x)

    st = {"case": dict(case)}
    kind, t = case["kind"], case["t"]
    if kind in ("swiglu", "swiglu_train"):
        h, i = case["h"], case["i"]
        st["x"] = normal(t, h).to(dt)
        st["w_gate"] = normal(i, h, std=0.02).to(dt)
        st["w_up"] = normal(i, h, std=0.02).to(dt)
        if kind == "swiglu_train":
            st["dh"] = normal(t, i, std=0.1).to(dt)
    elif kind == "int8":
        st["q"], st["s"] = _quant_rows(tokens(t, case["k"]))
        st["w_q"], st["w_s"] = _quant_rows(normal(case["n"], case["k"], std=0.02))
        st["bias"] = normal(case["n"], std=0.1) if case["bias"] else None
    elif kind == "int8_block":
        h = case["h"]
        st["res"] = tokens(t, h).to(dt)
        st["w_pre"] = (1 + normal(h, std=0.1)).to(dt)
        st["w_post"] = (1 + normal(h, std=0.1)).to(dt)
        st["w_q"], st["w_s"] = _quant_rows(normal(h, h, std=0.02))
        st["alpha"] = 0.5
    else:
        h = case["h"]
        st["res"] = tokens(t, h).to(dt)
        st["y"] = normal(t, h, std=0.5).to(dt)
        st["w_pre"] = (1 + normal(h, std=0.1)).to(dt)
        st["w_post"] = (1 + normal(h, std=0.1)).to(dt)
        shape = {"none": None, "channel": (h,), "token": (t, 1), "element": (t, h)}[case["gate"]]
        st["gate"] = None if shape is None else torch.sigmoid(normal(*shape)).to(dt)
        st["alpha"] = 0.5
        if kind == "norm_train":
            st["dr"] = normal(t, h, std=0.1).to(dt)
            st["dn"] = normal(t, h, std=0.1).to(dt)
    return st


def _quant_rows(x):
    """Symmetric INT8 codes of each row and the row's fp32 scale."""
    s = x.abs().amax(dim=1) / 127
    q = torch.where(s[:, None] > 0, x / s[:, None], torch.zeros_like(x)).round().clamp(-127, 127)
    return q.to(torch.int8), s


def run(st):
    return (_run_own if own else _run_plain)(st)


# ------------------------------------------------------------------ library calls
def _run_own(st):
    import int4_group_quantized_g128_amd as q4
    case = st["case"]
    kind = case["kind"]
    if kind == "swiglu":
        return q4.swiglu_linear_forward(st["x"], st["w_gate"], st["w_up"])
    if kind == "swiglu_train":
        h, gu = q4.swiglu_linear_forward(st["x"], st["w_gate"], st["w_up"], save=True)
        return (h,) + tuple(q4.swiglu_linear_backward(st["dh"], st["x"], st["w_gate"], st["w_up"], gu))
    if kind == "int8":
        return q4.int8_linear_forward(st["q"], st["s"], st["w_q"], st["w_s"], bias=st["bias"],
                                      out_dtype=DTYPES[case["dtype"]])
    if kind == "int8_block":
        q, s = q4.block_norm_forward(st["res"], w_pre=st["w_pre"], eps=EPS, quantize=True)[1:]
        y = q4.int8_linear_forward(q, s, st["w_q"], st["w_s"], out_dtype=st["res"].dtype)
        return q4.block_norm_forward(st["res"], y=y, w_post=st["w_post"], alpha=st["alpha"], eps=EPS)[0]
    args = dict(y=st["y"], w_post=st["w_post"], gate=st["gate"], alpha=st["alpha"], w_pre=st["w_pre"], eps=EPS)
    r, n = q4.block_norm_forward(st["res"], **args)
    if kind == "norm":
        return r, n
    g = q4.block_norm_backward(st["dr"], st["dn"], st["res"], **args)
    return r, n, g["res"], g["y"], g["w_post"], g["w_pre"], g["gate"]


# ------------------------------------------------------------------ plain form
def _int_product(q, w_q):
    """Exact integer sums q w_q^T as fp32 products over 1024 columns at a time: each
    partial sum stays within 2^24, and the partial sums are added as integers."""
    acc = None
    for k0 in range(0, q.shape[1], 1024):
        part = (q[:, k0:k0 + 1024].float() @ w_q[:, k0:k0 + 1024].float().t()).to(torch.int32)
        acc = part if acc is None else acc + part
    return acc


def _plain_int8(q, s, w_q, w_s, bias):
    y = _int_product(q, w_q).float() * (s[:, None] * w_s[None, :])
    return y if bias is None else y + bias


def _plain_norm(v, w):
    return v * torch.rsqrt((v * v).mean(dim=1, keepdim=True) + EPS) * w


def _plain_norm_grad(v, w, d):
    """Gradients of _plain_norm to v and, summed over rows, to w."""
    rstd = torch.rsqrt((v * v).mean(dim=1, keepdim=True) + EPS)
    vhat = v * rstd
    wd = w * d
    return rstd * (wd - vhat * (wd * vhat).mean(dim=1, keepdim=True)), (d * vhat).sum(dim=0)


def _run_plain(st):
    case = st["case"]
    kind, dt = case["kind"], DTYPES[case["dtype"]]
    if kind in ("swiglu", "swiglu_train"):
        x, wg, wu = st["x"].float(), st["w_gate"].float(), st["w_up"].float()
        g, u = x @ wg.t(), x @ wu.t()
        sig = 1 / (1 + torch.exp(-g))
        h = (g * sig * u).to(dt)
        if kind == "swiglu":
            return h
        dh = st["dh"].float()
        dg = dh * u * sig * (1 + g * (1 - sig))
        du = dh * g * sig
        return h, (dg @ wg + du @ wu).to(dt), (dg.t() @ x).to(dt), (du.t() @ x).to(dt)
    if kind == "int8":
        return _plain_int8(st["q"], st["s"], st["w_q"], st["w_s"], st["bias"]).to(dt)
    if kind == "int8_block":
        res = st["res"].float()
        n = _plain_norm(res, st["w_pre"].float())
        q, s = _quant_rows(n)
        y = _plain_int8(q, s, st["w_q"], st["w_s"], None).to(dt).float()
        return (res + st["alpha"] * _plain_norm(y, st["w_post"].float())).to(dt)
    res, y = st["res"].float(), st["y"].float()
    w_post, w_pre, alpha = st["w_post"].float(), st["w_pre"].float(), st["alpha"]
    gate = None if st["gate"] is None else st["gate"].float()
    p = _plain_norm(y, w_post)
    r = res + alpha * (p if gate is None else gate * p)
    n = _plain_norm(r, w_pre)
    if kind == "norm":
        return r.to(dt), n.to(dt)
    d, dw_pre = _plain_norm_grad(r, w_pre, st["dn"].float())
    dres = st["dr"].float() + d
    e = alpha * dres
    dy, dw_post = _plain_norm_grad(y, w_post, e if gate is None else e * gate)
    dgate = None
    if gate is not None:
        dgate = e * p
        if case["gate"] == "channel":
            dgate = dgate.sum(dim=0)
        elif case["gate"] == "token":
            dgate = dgate.sum(dim=1, keepdim=True)
        else:
            dgate = dgate.to(dt)
    return r.to(dt), n.to(dt), dres.to(dt), dy.to(dt), dw_post, dw_pre, dgate


# ------------------------------------------------------------------ work and exact values
def work(case):
    t, e = case["t"], 4 if case["dtype"] == "fp32" else 2
    kind = case["kind"]
    if kind in ("swiglu", "swiglu_train"):
        h, i = case["h"], case["i"]
        if kind == "swiglu":
            return {"bytes": e * (t * h + 2 * i * h + t * i), "flops": 4 * t * h * i}
        # x, both weights and dh in; h, dx and both weight gradients out
        return {"bytes": e * (2 * t * h + 4 * i * h + 2 * t * i), "flops": 12 * t * h * i}
    if kind == "int8":
        k, n = case["k"], case["n"]
        return {"bytes": t * k + n * k + 4 * (t + n) + e * t * n + (4 * n if case["bias"] else 0),
                "flops": 2 * t * n * k}
    if kind == "int8_block":
        h = case["h"]
        return {"bytes": e * 2 * t * h + h * h + 4 * h + 2 * e * h, "flops": 2 * t * h * h}
    h = case["h"]
    gate = {"none": 0, "channel": h, "token": t, "element": t * h}[case["gate"]]
    if kind == "norm":
        return {"bytes": e * (4 * t * h + 2 * h + gate), "flops": 10 * t * h}
    # res, y, dr, dn in; r, n, dres, dy and the gradients of the weights and the gate out
    dgate = e * gate if case["gate"] == "element" else 4 * gate
    return {"bytes": e * (8 * t * h + 2 * h + gate) + 8 * h + dgate, "flops": 35 * t * h}


def exact(case, seed):
    st = prepare(case, seed)
    kind = case["kind"]
    d = {k: v.double() for k, v in st.items() if isinstance(v, torch.Tensor)}

    def unit(v):
        """v over its root mean square, and the inverse of that root."""
        inv = (v.square().sum(1, keepdim=True) / v.shape[1] + EPS).pow(-0.5)
        return v * inv, inv

    if kind in ("swiglu", "swiglu_train"):
        a = torch.matmul(d["x"], d["w_gate"].T)
        b = torch.matmul(d["x"], d["w_up"].T)
        sg = torch.sigmoid(a)
        act = a * sg
        if kind == "swiglu":
            return act * b
        da = d["dh"] * b * (sg + act * (1 - sg))
        db = d["dh"] * act
        dx = torch.matmul(da, d["w_gate"]) + torch.matmul(db, d["w_up"])
        return act * b, dx, torch.matmul(da.T, d["x"]), torch.matmul(db.T, d["x"])
    if kind == "int8":
        y = torch.matmul(d["q"], d["w_q"].T) * d["s"].reshape(-1, 1) * d["w_s"].reshape(1, -1)
        return y + d["bias"] if case["bias"] else y
    if kind == "int8_block":
        n = unit(d["res"])[0] * d["w_pre"]
        s = n.abs().amax(1, keepdim=True) / 127
        q = torch.where(s > 0, torch.round(n / s), torch.zeros_like(n))
        y = torch.matmul(q, d["w_q"].T) * s * d["w_s"].reshape(1, -1)
        y = y.to(st["res"].dtype).double()   # the block's output, in the stream's type
        return d["res"] + st["alpha"] * unit(y)[0] * d["w_post"]
    alpha = st["alpha"]
    gate = torch.ones((), dtype=torch.float64, device="cuda") if st["gate"] is None else d["gate"]
    yh, yi = unit(d["y"])
    p = yh * d["w_post"]
    r = d["res"] + alpha * gate * p
    rh, ri = unit(r)
    n = rh * d["w_pre"]
    if kind == "norm":
        return r, n
    back = lambda vh, inv, c: inv * (c - vh * (c * vh).sum(1, keepdim=True) / vh.shape[1])
    dr = d["dr"] + back(rh, ri, d["dn"] * d["w_pre"])
    dp = alpha * gate * dr
    dy = back(yh, yi, dp * d["w_post"])
    dg = alpha * dr * p
    dg = {"none": lambda: None, "channel": lambda: dg.sum(0), "token": lambda: dg.sum(1, keepdim=True),
          "element": lambda: dg}[case["gate"]]()
    return r, n, dr, dy, (dp * yh).sum(0), (d["dn"] * rh).sum(0), dg
