"""Cases of the FP8 experts and the token order around them, in plain form and as library calls.

* moe_dispatch / moe_combine: tokens sorted by expert and back with their weights, and the
  gradients of both;
* fp8_linear: the e4m3 product with a scale for each block of 128, for one matrix and for the
  experts of a layer (rows grouped by expert), forward and backward, with its quantisers;
* the experts block: tokens -> sorted e4m3 codes -> gate and up projection -> silu(g) u in e4m3
  -> down projection -> weighted sum per token.

``own`` selects what ``run`` does: False, elementary torch operations in 32 bits; True, the
library's entry points.
"""
import math

import torch

own = False

BLOCK = 128
E4M3 = torch.float8_e4m3fn
E4M3_MAX = 448.0
DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}


def listed():
    return [
        # one decoded token to its eight experts and back, in a layer of 256 experts
        dict(name="tokens_t1", kind="tokens", t=1, h=7168, k=8, e=256, first=0, held=256, dtype="bf16"),
        # a prefill chunk through the same layer
        dict(name="tokens_t4096", kind="tokens", t=4096, h=7168, k=8, e=256, first=0, held=256, dtype="bf16"),
        # a training step of the 8-expert, top-2 layer: both directions and their gradients
        dict(name="tokens_train_t4096", kind="tokens_train", t=4096, h=2048, k=2, e=8, first=0, held=8, dtype="bf16"),
        # an odd batch and width in fp16 on a rank that holds 24 of 40 experts
        dict(name="tokens_train_ragged", kind="tokens_train", t=777, h=1001, k=6, e=40, first=8, held=24, dtype="fp16"),
        # one token through the stacked gate and up projections of a 2048 / 8192 dense FFN
        dict(name="fp8_t1", kind="fp8", t=1, k=2048, n=16384, dtype="bf16"),
        # a decode batch through the shared expert's gate and up projections (7168 / 2048)
        dict(name="fp8_t64", kind="fp8", t=64, k=7168, n=4096, dtype="bf16"),
        # a prefill chunk through the same
        dict(name="fp8_t4096", kind="fp8", t=4096, k=7168, n=4096, dtype="bf16"),
        # odd lengths and a width that no block divides, in fp16
        dict(name="fp8_ragged", kind="fp8", t=333, k=1040, n=1001, dtype="fp16"),
        # a training step of the dense FFN's gate and up projections
        dict(name="fp8_train_t4096", kind="fp8_train", t=4096, k=2048, n=16384, dtype="bf16"),
        # a decode batch through a rank's 32 of 256 experts
        dict(name="experts_t64", kind="experts", t=64, h=7168, i=2048, k=8, e=256, first=64, held=32, dtype="bf16"),
        # a prefill chunk through them
        dict(name="experts_t4096", kind="experts", t=4096, h=7168, i=2048, k=8, e=256, first=64, held=32, dtype="bf16"),
        # a training step of the 8-expert layer's gate and up projections, rows sorted by expert
        dict(name="experts_train_t4096", kind="experts_train", t=4096, h=2048, n=2048, k=2, e=8, first=0, held=8,
             dtype="bf16"),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _width(rng, lo, hi, step):
    """A width between lo and hi, a multiple of step; one in two a multiple of 128."""
    w = _log_int(rng, lo, hi)
    step = 128 if rng.random() < 0.5 else step
    return max(step, w // step * step)


def _experts(rng, most):
    """k choices of e experts, of which a rank holds `held` from `first` on."""
    e = _log_int(rng, 1, 256)
    k = rng.randint(1, min(e, 8))
    held = e if rng.random() < 0.5 else rng.randint(1, e)
    held = min(held, most)
    return dict(k=k, e=e, first=rng.randint(0, e - held), held=held)


def draw(rng):
    kind = rng.choice(["tokens", "tokens_train", "fp8", "fp8", "fp8_train", "experts", "experts_train"])
    t = _log_int(rng, 1, 4096)
    if kind in ("tokens", "tokens_train"):
        c = dict(kind=kind, t=t, h=_log_int(rng, 64, 7168), dtype=rng.choice(["bf16", "fp16", "fp32"]),
                 **_experts(rng, 256))
        if rng.random() < 0.5:
            c["h"] = c["h"] // 8 * 8
        while kind == "tokens_train" and c["t"] * c["k"] * c["h"] > 4096 * 2 * 7168:
            c["t"] = (c["t"] + 1) // 2
        return c
    if kind == "fp8":
        k, n = _width(rng, 64, 8192, 16), _log_int(rng, 16, 16384)
        while t * k * n > 4096 * 2048 * 16384:
            t = (t + 1) // 2
        return dict(kind=kind, t=t, k=k, n=n, dtype=rng.choice(["bf16", "fp16"]))
    if kind == "fp8_train":
        k, n = _width(rng, 64, 8192, 16), _width(rng, 64, 16384, 16)
        while t * k * n > 4096 * 2048 * 16384:
            t = (t + 1) // 2
        return dict(kind=kind, t=t, k=k, n=n, dtype=rng.choice(["bf16", "fp16"]))
    if kind == "experts":
        return dict(kind=kind, t=t, h=_width(rng, 64, 7168, 16), i=_width(rng, 64, 2048, 16),
                    dtype=rng.choice(["bf16", "fp16"]), **_experts(rng, 32))
    return dict(kind=kind, t=t, h=_width(rng, 64, 4096, 16), n=_width(rng, 64, 2048, 16),
                dtype=rng.choice(["bf16", "fp16"]), **_experts(rng, 16))


# ------------------------------------------------------------------ inputs
def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(int(seed))
    dt = DTYPES[case["dtype"]]
    kind, t = case["kind"], case["t"]

    def normal(*shape, std=1.0):
        return torch.randn(*shape, generator=gen, device="cuda") * std

    def tokens(rows, w):
        # unit tokens with 1 % of the channels ten times larger, as hidden states have them
        x = normal(rows, w)
        big = torch.rand(w, generator=gen, device="cuda") < 0.01
        return torch.where(big, x * 10, x)

    def gradient(rows, w):
        # rows of different sizes, as the losses of different tokens make them
        return normal(rows, w) * (0.01 * torch.exp(normal(rows, 1)))

    st = {"case": dict(case)}
    if "e" in case:
        # experts of unequal popularity, the weights a softmax over the chosen
        score = normal(t, case["e"]) + normal(case["e"], std=0.7)
        top, ids = score.topk(case["k"], dim=1)
        st["ids"] = ids.to(torch.int32).contiguous()
        st["weights"] = torch.softmax(top, dim=1).contiguous()
        local = st["ids"].long() - case["first"]
        local = local[(local >= 0) & (local < case["held"])]
        counts = torch.bincount(local, minlength=case["held"])
        st["most"] = max(1, int(counts.max()))   # the plain form's room per expert
    if kind in ("tokens", "tokens_train"):
        h, p = case["h"], t * case["k"]
        st["x"] = tokens(t, h).to(dt)
        st["y"] = normal(p, h, std=0.5).to(dt)
        if kind == "tokens_train":
            st["dxp"] = gradient(p, h).to(dt)
            st["dout"] = gradient(t, h).to(dt)
        if case["held"] < case["e"]:   # rows that no slot takes keep what these hold
            st["xp_out"] = torch.zeros(p, h, dtype=dt, device="cuda")
            if kind == "tokens_train":
                st["dy_out"] = torch.zeros(p, h, dtype=dt, device="cuda")
    elif kind in ("fp8", "fp8_train"):
        st["x"] = tokens(t, case["k"]).to(dt)
        st["w_q"], st["w_s"] = _weight_codes(normal(case["n"], case["k"], std=0.02))
        if kind == "fp8_train":
            st["dy"] = gradient(t, case["n"]).to(dt)
    elif kind == "experts":
        h, i, held = case["h"], case["i"], case["held"]
        st["x"] = tokens(t, h).to(dt)
        st["gu_q"], st["gu_s"] = _weight_codes(normal(held, 2 * i, h, std=0.02))
        st["dn_q"], st["dn_s"] = _weight_codes(normal(held, h, i, std=0.02))
    else:
        h, n, held = case["h"], case["n"], case["held"]
        st["x"] = tokens(t, h).to(dt)
        st["w_q"], st["w_s"] = _weight_codes(normal(held, n, h, std=0.02))
        st["dy"] = gradient(t * case["k"], n).to(dt)
        if held < case["e"]:
            st["xp_out"] = torch.zeros(t * case["k"], h, dtype=dt, device="cuda")
            st["y_out"] = torch.zeros(t * case["k"], n, dtype=dt, device="cuda")
            st["dx_out"] = torch.zeros(t * case["k"], h, dtype=dt, device="cuda")
    return st


def _weight_codes(w):
    """e4m3 codes of the last two axes' 128 x 128 blocks and the blocks' scales."""
    b = _blocks(w)
    s = _scale(b.abs().amax(dim=(-3, -1)))
    d = s[..., :, None, :, None]
    q = torch.where(d > 0, b / d, torch.zeros_like(b)).clamp_(-E4M3_MAX, E4M3_MAX).to(E4M3)
    n, k = w.shape[-2:]
    return q.flatten(-2).flatten(-3, -2)[..., :n, :k].contiguous(), s


def _scale(most):
    """The fp32 quotient by 448 (by a tensor: torch multiplies by the inverse of a number)."""
    return most / torch.full_like(most, E4M3_MAX)


def _blocks(w):
    """[.., n, k] as [.., n / 128, 128, k / 128, 128], padded with zeros."""
    n, k = w.shape[-2:]
    w = torch.nn.functional.pad(w, (0, -k % BLOCK, 0, -n % BLOCK))
    return w.unflatten(-1, (-1, BLOCK)).unflatten(-3, (-1, BLOCK))


def run(st):
    return (_run_own if own else _run_plain)(st)


# ------------------------------------------------------------------ library calls
def _run_own(st):
    import int4_group_quantized_g128_amd as q4
    case = st["case"]
    kind, dt = case["kind"], DTYPES[case["dtype"]]
    if kind in ("tokens", "tokens_train"):
        xp, offsets, perm, inv = q4.moe_dispatch_forward(st["x"], st["ids"], case["held"], first=case["first"],
                                                         out=st.get("xp_out"))
        out = q4.moe_combine_forward(st["y"], inv, st["weights"])
        if kind == "tokens":
            return xp, offsets, perm, inv, out
        dx = q4.moe_dispatch_backward(st["dxp"], inv)
        dy, dw = q4.moe_combine_backward(st["dout"], st["y"], inv, st["weights"], out=st.get("dy_out"))
        return xp, offsets, perm, inv, out, dx, dy, dw
    if kind == "fp8":
        q, s = q4.quantize_fp8_tokens(st["x"])
        return q4.fp8_linear_forward(q, s, st["w_q"], st["w_s"], out_dtype=dt)
    if kind == "fp8_train":
        q, s, qc, sc = q4.quantize_fp8_tokens(st["x"], columns=True)
        y = q4.fp8_linear_forward(q, s, st["w_q"], st["w_s"], out_dtype=dt)
        dx, dw = q4.fp8_linear_backward(st["dy"], qc, sc, st["w_q"], st["w_s"])
        return y, dx, dw
    if kind == "experts":
        q, s, offsets, perm, inv = q4.moe_dispatch_forward(st["x"], st["ids"], case["held"], first=case["first"],
                                                           quantize=True)
        gu = q4.fp8_linear_forward(q, s, st["gu_q"], st["gu_s"], offsets=offsets, out_dtype=dt)
        q, s = q4.quantize_fp8_tokens(gu, gated=True, offsets=offsets)
        y = q4.fp8_linear_forward(q, s, st["dn_q"], st["dn_s"], offsets=offsets, out_dtype=dt)
        return q4.moe_combine_forward(y, inv, st["weights"])
    xp, offsets, perm, inv = q4.moe_dispatch_forward(st["x"], st["ids"], case["held"], first=case["first"],
                                                     out=st.get("xp_out"))
    q, s, qc, sc = q4.quantize_fp8_tokens(xp, columns=True, offsets=offsets)
    y = q4.fp8_linear_forward(q, s, st["w_q"], st["w_s"], offsets=offsets, out_dtype=dt, out=st.get("y_out"))
    dxp, dw = q4.fp8_linear_backward(st["dy"], qc, sc, st["w_q"], st["w_s"], offsets=offsets, out=st.get("dx_out"))
    return y, dxp, dw, q4.moe_dispatch_backward(dxp, inv)


# ------------------------------------------------------------------ plain form
def _sorted(ids, first, held):
    """Slots sorted by expert, those of other ranks' experts last: offsets, perm and inv, with
    -1 for what is not held, and each position's expert (held: none)."""
    p = ids.numel()
    local = ids.reshape(-1).long() - first
    local = torch.where((local >= 0) & (local < held), local, held)
    key = torch.sort(local * p + torch.arange(p, device=ids.device)).values
    expert, perm = key // p, key % p
    offsets = (local[None, :] < torch.arange(held + 1, device=ids.device)[:, None]).sum(dim=1)
    pos = torch.arange(p, device=ids.device)
    inv = torch.empty_like(perm)
    inv[perm] = torch.where(expert < held, pos, -1)
    return offsets, torch.where(expert < held, perm, -1), inv.reshape(ids.shape), expert


def _dispatch(x, perm, k):
    return torch.where(perm[:, None] >= 0, x[perm.clamp(min=0) // k], 0)


def _combine(y, inv, weights):
    """Sums of a token's rows (times its weights), a row that it lacks as zero."""
    rows = torch.where(inv[:, :, None] >= 0, y[inv.clamp(min=0)], 0)
    return (rows if weights is None else rows * weights[:, :, None]).sum(dim=1)


def _codes(groups, dims):
    """What e4m3 codes with one scale over `dims` stand for."""
    s = _scale(groups.abs().amax(dim=dims, keepdim=True))
    q = torch.where(s > 0, groups / s, torch.zeros_like(groups)).clamp(-E4M3_MAX, E4M3_MAX)
    return q.to(E4M3).float() * s


def _row_codes(x):
    """Groups of 128 along the last axis."""
    k = x.shape[-1]
    g = torch.nn.functional.pad(x, (0, -k % BLOCK)).unflatten(-1, (-1, BLOCK))
    return _codes(g, -1).flatten(-2)[..., :k]


def _column_codes(x):
    """Groups of 128 along the last axis but one."""
    t = x.shape[-2]
    g = torch.nn.functional.pad(x, (0, 0, 0, -t % BLOCK)).unflatten(-2, (-1, BLOCK))
    return _codes(g, -2).flatten(-3, -2)[..., :t, :]


def _weights(q, s):
    n, k = q.shape[-2:]
    b = _blocks(q.float()) * s[..., :, None, :, None]
    return b.flatten(-2).flatten(-3, -2)[..., :n, :k]


def _silu_up(gu):
    g, u = gu.chunk(2, dim=-1)
    return g / (1 + torch.exp(-g)) * u


def _by_expert(rows, place, held, most):
    """Rows [p, w] as [held, most, w], zeros where an expert has fewer (place: a row's index)."""
    out = torch.zeros(held * most + 1, rows.shape[1], device=rows.device)
    out[place] = rows
    return out[:-1].unflatten(0, (held, most))


def _run_plain(st):
    case = st["case"]
    kind, dt = case["kind"], DTYPES[case["dtype"]]
    if kind in ("fp8", "fp8_train"):
        x, w = st["x"].float(), _weights(st["w_q"], st["w_s"])
        y = (_row_codes(x) @ w.t()).to(dt)
        if kind == "fp8":
            return y
        dy = st["dy"].float()
        return y, (_row_codes(dy) @ w).to(dt), (_column_codes(dy).t() @ _column_codes(x)).to(dt)
    k, held, most = case["k"], case["held"], st["most"]
    offsets, perm, inv, expert = _sorted(st["ids"], case["first"], held)
    xp = _dispatch(st["x"].float(), perm, k)
    order = (offsets.int(), perm.int(), inv.int())
    if kind in ("tokens", "tokens_train"):
        y, w = st["y"].float(), st["weights"]
        out = _combine(y, inv, w).to(dt)
        if kind == "tokens":
            return (xp.to(dt),) + order + (out,)
        dout = st["dout"].float()
        wp = torch.where(perm >= 0, w.reshape(-1)[perm.clamp(min=0)], 0)
        dy = wp[:, None] * _dispatch(dout, perm, k)
        own_rows = torch.where(inv[:, :, None] >= 0, y[inv.clamp(min=0)], 0)
        dw = (own_rows * dout[:, None, :]).sum(dim=2)
        return (xp.to(dt),) + order + (out, _combine(st["dxp"].float(), inv, None).to(dt), dy.to(dt), dw)
    rank = torch.arange(perm.numel(), device=perm.device) - offsets[expert.clamp(max=held)]
    place = torch.where(expert < held, expert * most + rank, held * most)
    unpad = lambda v: torch.nn.functional.pad(v.flatten(0, 1), (0, 0, 0, 1))[place]
    xe = _by_expert(xp, place, held, most)
    if kind == "experts":
        gu = torch.bmm(_row_codes(xe), _weights(st["gu_q"], st["gu_s"]).transpose(1, 2).contiguous())
        h = _row_codes(_silu_up(gu.to(dt).float()))
        y = torch.bmm(h, _weights(st["dn_q"], st["dn_s"]).transpose(1, 2).contiguous())
        return _combine(unpad(y).to(dt).float(), inv, st["weights"]).to(dt)
    w = _weights(st["w_q"], st["w_s"])
    y = unpad(torch.bmm(_row_codes(xe), w.transpose(1, 2).contiguous())).to(dt)
    de = _by_expert(st["dy"].float(), place, held, most)
    dxp = unpad(torch.bmm(_row_codes(de), w)).to(dt)
    dw = torch.bmm(_column_codes(de).transpose(1, 2).contiguous(), _column_codes(xe))
    return y, dxp, dw.to(dt), _combine(dxp.float(), inv, None).to(dt)


# ------------------------------------------------------------------ work and exact values
def _held_rows(case):
    """Rows that a rank's experts get where tokens choose evenly."""
    return max(1, case["t"] * case["k"] * case["held"] // case["e"])


def work(case):
    kind, t, z = case["kind"], case["t"], 4 if case["dtype"] == "fp32" else 2
    if kind in ("tokens", "tokens_train"):
        h, k, p = case["h"], case["k"], _held_rows(case)
        # x, y and the choices in; the sorted rows, the order and the sums out
        b = z * h * (2 * t + 2 * p) + t * k * 16
        f = 2 * p * h
        if kind == "tokens_train":   # dxp, dout and y in; dx, dy and the weights' gradients out
            b += z * h * (2 * t + 2 * p) + t * k * 4
            f += 4 * p * h
        return {"bytes": b, "flops": f}
    if kind in ("fp8", "fp8_train"):
        k, n = case["k"], case["n"]
        b = z * t * k + n * k + z * t * n
        if kind == "fp8":
            return {"bytes": b, "flops": 2 * t * n * k}
        return {"bytes": b + z * t * n + z * t * k + z * n * k, "flops": 6 * t * n * k}
    p, held = _held_rows(case), case["held"]
    hit = min(held, p)   # experts with a row, at most
    if kind == "experts":
        h, i = case["h"], case["i"]
        return {"bytes": 2 * z * t * h + hit * 3 * h * i + t * case["k"] * 8, "flops": 6 * p * h * i}
    h, n = case["h"], case["n"]
    return {"bytes": z * (2 * t * h + p * h + 2 * p * n) + hit * n * h + z * held * n * h, "flops": 6 * p * n * h}


def exact(case, seed):
    st = prepare(case, seed)
    kind, dt = case["kind"], DTYPES[case["dtype"]]

    def e4m3(v, axis):
        """v (64 bits) as codes times scales, groups of 128 along `axis`; the scale and the
        quotient are fp32 numbers by definition (64 bits hold them before that rounding)."""
        v = v.transpose(axis, -1)
        out = torch.zeros_like(v)
        for a in range(0, v.shape[-1], BLOCK):
            g = v[..., a:a + BLOCK]
            s = (g.abs().max(dim=-1, keepdim=True).values / 448).float().double()
            c = torch.where(s > 0, (g / s).float().double(), 0.0 * g).clamp(-448, 448)
            out[..., a:a + BLOCK] = c.float().to(E4M3).double() * s
        return out.transpose(axis, -1)

    def full(q, s):
        big = s.double().repeat_interleave(BLOCK, -2).repeat_interleave(BLOCK, -1)
        return q.double() * big[..., :q.shape[-2], :q.shape[-1]]

    if kind in ("fp8", "fp8_train"):
        x, w = st["x"].double(), full(st["w_q"], st["w_s"])
        y = e4m3(x, 1) @ w.T
        if kind == "fp8":
            return y
        dy = st["dy"].double()
        return y, e4m3(dy, 1) @ w, e4m3(dy, 0).T @ e4m3(x, 0)
    # the order, token by token on the host
    k, held, t = case["k"], case["held"], case["t"]
    lists = [[] for _ in range(held)]
    for slot, expert in enumerate(st["ids"].reshape(-1).tolist()):
        if 0 <= expert - case["first"] < held:
            lists[expert - case["first"]].append(slot)
    flat = [slot for one in lists for slot in one]
    ends = [0]
    for one in lists:
        ends.append(ends[-1] + len(one))
    slots = torch.tensor(flat, dtype=torch.long, device="cuda")
    total, p = len(flat), t * k
    weights = st["weights"].double().reshape(-1)

    def gather(v):
        return v[slots // k]

    def back(rows, scaled):
        out = torch.zeros(t, rows.shape[1], dtype=torch.float64, device="cuda")
        return out.index_add_(0, slots // k, rows * weights[slots, None] if scaled else rows)

    def whole(rows):
        out = torch.zeros(p, rows.shape[1], dtype=torch.float64, device="cuda")
        out[:total] = rows
        return out

    if kind in ("tokens", "tokens_train"):
        y = st["y"].double()[:total]
        offsets = torch.tensor(ends, dtype=torch.int32, device="cuda")
        perm = torch.full((p,), -1, dtype=torch.int32, device="cuda")
        perm[:total] = slots.int()
        inv = torch.full((p,), -1, dtype=torch.int32, device="cuda")
        inv[slots] = torch.arange(total, dtype=torch.int32, device="cuda")
        res = (whole(gather(st["x"].double())), offsets, perm, inv.reshape(t, k), back(y, True))
        if kind == "tokens":
            return res
        dout = gather(st["dout"].double())
        dw = torch.zeros(p, dtype=torch.float64, device="cuda")
        dw[slots] = (dout * y).sum(1)
        return res + (back(st["dxp"].double()[:total], False), whole(dout * weights[slots, None]), dw.reshape(t, k))
    rows = gather(st["x"].double())

    def each(width, f):
        out = torch.zeros(total, width, dtype=torch.float64, device="cuda")
        for x in range(held):
            if ends[x + 1] > ends[x]:
                out[ends[x]:ends[x + 1]] = f(x, slice(ends[x], ends[x + 1]))
        return out

    if kind == "experts":
        i = case["i"]
        gu = each(2 * i, lambda x, at: e4m3(rows[at], 1) @ full(st["gu_q"][x], st["gu_s"][x]).T).to(dt).double()
        hid = gu[:, :i] * torch.sigmoid(gu[:, :i]) * gu[:, i:]
        # (the activation is an fp32 number before it is quantised)
        y = each(case["h"], lambda x, at: e4m3(hid[at].float().double(), 1) @ full(st["dn_q"][x], st["dn_s"][x]).T)
        return back(y.to(dt).double(), True)
    dy = st["dy"].double()[:total]
    y = each(case["n"], lambda x, at: e4m3(rows[at], 1) @ full(st["w_q"][x], st["w_s"][x]).T)
    dxp = each(case["h"], lambda x, at: e4m3(dy[at], 1) @ full(st["w_q"][x], st["w_s"][x]))
    dw = torch.zeros(held, case["n"], case["h"], dtype=torch.float64, device="cuda")
    for x in range(held):
        at = slice(ends[x], ends[x + 1])
        if ends[x + 1] > ends[x]:
            dw[x] = e4m3(dy[at], 0).T @ e4m3(rows[at], 0)
    return whole(y), whole(dxp), dw, back(dxp.to(dt).double(), False)
