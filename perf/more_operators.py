"""Timed cases of the 4-bit and the expert-grouped products beside a paged MoE layer.

A layer whose experts all stay in GPU memory, or whose experts are trained, runs
these: `group_rows` (the routed entries of pe.route's ids, ordered by expert),
`grouped_glu` and `grouped_linear` (each expert's product over its own rows, in
bf16, group-128 int4 or MXFP4), `combine` (each token's weighted sum of its
experts' rows), and for training `combine_backward` and `grouped_ffn_backward`.
`linear_w4` and `glu_w4` are the same 4-bit products for the always-on shared
expert or a dense layer.

`own` chooses between plain torch arithmetic in 32 bits and libpe's kernels.
Sizes: hidden 2048 and expert intermediate 768 with 128 experts, top-8, and
hidden and intermediate 2880 with 32 experts, top-4, are the workloads of
synth/workloads.py; an intermediate of 6144 is as wide as eight experts of 768
together; 2048 tokens is the prefill chunk.
"""
import math

import torch

own = False

DEV = "cuda"
E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0, -0.0, -0.5, -1.0, -1.5, -2.0, -3.0, -4.0, -6.0)


# ------------------------------------------------------------------ cases

def listed():
    return [
        # Down projection of a dense block for one decode token, added to the residual stream: the weights' bytes.
        dict(name="w4_linear_decode", op="linear_w4", wtype="int4", T=1, N=2048, K=6144, bias=False, residual=True,
             act="none", out="bf16"),
        # Gate/up of a shared expert in the MXFP4 workload's shape for four requests.
        dict(name="w4_glu_decode", op="glu_w4", wtype="mxfp4", T=4, H=2880, I=2880, act="silu"),
        # The dense block's down projection over a prefill chunk.
        dict(name="w4_linear_prefill", op="linear_w4", wtype="int4", T=2048, N=2048, K=6144, bias=False, residual=True,
             act="none", out="bf16"),
        # Order by expert of a decode step's entries: four requests, 128 experts, top-8.
        dict(name="rows_decode", op="rows", T=4, E=128, k=8, skew=0.5),
        # The same for a long prefill.
        dict(name="rows_prefill", op="rows", T=8192, E=128, k=8, skew=0.5),
        # Gate/up of the routed experts for that decode step, int4: some 30 experts with a row or two each.
        dict(name="grouped_glu_decode", op="grouped_glu", wtype="int4", T=4, E=128, k=8, H=2048, I=768, act="silu",
             save=False, skew=0.5),
        # Gate/up over a prefill chunk in bf16, keeping what the backward pass needs.
        dict(name="grouped_glu_prefill", op="grouped_glu", wtype="bf16", T=2048, E=128, k=8, H=2048, I=768, act="silu",
             save=True, skew=0.5),
        # Down projection with bias of MXFP4 experts, an odd number of tokens.
        dict(name="grouped_linear_odd", op="grouped_linear", wtype="mxfp4", T=1023, E=32, k=4, N=2880, K=2880, bias=True,
             skew=0.5),
        # Gradients of eight experts over a short, odd batch.
        dict(name="grouped_backward_small", op="grouped_backward", T=257, E=8, k=2, H=2048, I=768, act="silu", skew=0.5),
        # Gradients of a whole layer's experts over a chunk of 2048 tokens.
        dict(name="grouped_backward_large", op="grouped_backward", T=2048, E=128, k=8, H=2048, I=768, act="silu",
             skew=0.5),
        # Weighted sum of the experts' outputs of a long prefill, added to the residual stream.
        dict(name="combine_prefill", op="combine", T=8192, k=8, H=2048, residual=True),
        # Its gradients, an odd number of tokens of the MXFP4 workload's width.
        dict(name="combine_backward_odd", op="combine_backward", T=1023, k=4, H=2880),
    ]


def _log(rng, lo, hi, step=1):
    """An integer in [lo, hi], spread over its logarithm, a multiple of `step`."""
    v = math.exp(rng.uniform(math.log(lo), math.log(hi + 0.999)))
    return max(lo, min(hi, int(v) // step * step))


def draw(rng):
    op = rng.choice(["linear_w4", "glu_w4", "rows", "grouped_glu", "grouped_linear", "grouped_backward", "combine",
                     "combine_backward"])
    if op in ("linear_w4", "glu_w4"):
        wtype = rng.choice(["int4", "mxfp4"])
        step = 128 if wtype == "int4" else 32
        T, K = _log(rng, 1, 4096), _log(rng, 128, 6144, step)
        if op == "glu_w4":
            return dict(op=op, wtype=wtype, T=T, H=K, I=_log(rng, 128, 6144, 8), act=rng.choice(["silu", "gelu"]))
        return dict(op=op, wtype=wtype, T=T, N=_log(rng, 16, 6144), K=K, bias=rng.random() < 0.5,
                    residual=rng.random() < 0.5, act=rng.choice(["none", "silu", "gelu"]),
                    out=rng.choice(["bf16", "fp32"]))
    E, skew = _log(rng, 4, 128), rng.choice([0.0, 0.5, 1.0])
    k = rng.randint(1, min(E, 8))
    if op == "rows":
        return dict(op=op, T=_log(rng, 1, 8192), E=E, k=k, skew=skew)
    if op in ("combine", "combine_backward"):
        c = dict(op=op, T=_log(rng, 1, 8192), k=k, H=_log(rng, 128, 2880, 8))
        return dict(c, residual=rng.random() < 0.5) if op == "combine" else c
    if op == "grouped_backward":
        return dict(op=op, T=_log(rng, 1, 2048), E=E, k=k, H=_log(rng, 128, 2048, 8), I=_log(rng, 64, 768, 8),
                    act=rng.choice(["silu", "gelu"]), skew=skew)
    wtype = rng.choice(["bf16", "int4", "mxfp4"])
    T, K = _log(rng, 1, 2048), _log(rng, 128, 2880, {"bf16": 8, "int4": 128, "mxfp4": 32}[wtype])
    if op == "grouped_glu":
        return dict(op=op, wtype=wtype, T=T, E=E, k=k, H=K, I=_log(rng, 64, 1536, 8), act=rng.choice(["silu", "gelu"]),
                    save=wtype == "bf16" and rng.random() < 0.5, skew=skew)
    return dict(op=op, wtype=wtype, T=T, E=E, k=k, N=_log(rng, 64, 2880), K=K, bias=rng.random() < 0.5, skew=skew)


# ------------------------------------------------------------------ inputs

def _quantise(w, wtype):
    """Codes (two to a byte, the even column low) and scales of weights whose last dimension is summed over."""
    size = 128 if wtype == "int4" else 32
    b = w.view(*w.shape[:-1], w.shape[-1] // size, size)
    top = b.abs().amax(-1, keepdim=True)
    if wtype == "int4":
        s = (top / 7.5).clamp_min(2.0 ** -14).to(torch.float16)
        q = (torch.round(b / s.float()) + 8).clamp(0, 15)
        scales = s.squeeze(-1)
    else:
        e = torch.floor(torch.log2(top.clamp_min(2.0 ** -100))) - 2
        v = (b / torch.exp2(e)).clamp(-6, 6)
        edges = torch.tensor([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0], device=w.device)
        q = torch.bucketize(v.abs(), edges) + 8 * (v < 0)
        scales = (e + 127).squeeze(-1).to(torch.uint8)
    q = q.reshape(w.shape).to(torch.uint8)
    return (q[..., 0::2] | q[..., 1::2] << 4).contiguous(), scales.contiguous()


def _routed(T, E, k, skew, g):
    """int32 ids [T, k], distinct in each row, some experts more popular than others."""
    score = torch.randn((T, E), generator=g, device=DEV) + skew * torch.randn(E, generator=g, device=DEV)
    return score.topk(k, dim=1).indices.to(torch.int32).contiguous()


def _grouping(ids, E):
    """Offsets of the experts, the tokens in their order and the place of each entry."""
    flat = ids.reshape(-1)
    entries = torch.sort(flat, stable=True).indices
    places = torch.empty_like(entries)
    places[entries] = torch.arange(entries.numel(), device=DEV)
    offsets = (flat[None, :] < torch.arange(E + 1, device=DEV)[:, None]).sum(1)
    rows = torch.div(entries, ids.shape[1], rounding_mode="floor")
    return offsets.to(torch.int32), rows.to(torch.int32), places.view(ids.shape).to(torch.int32)


def prepare(case, seed):
    g = torch.Generator(device=DEV).manual_seed(seed)

    def rnd(*shape, std=1.0, dtype=torch.bfloat16):
        return (torch.randn(shape, generator=g, device=DEV) * std).to(dtype)

    def empty(*shape, dtype=torch.bfloat16):
        return torch.empty(shape, dtype=dtype, device=DEV)

    def weights(*shape):
        w = torch.randn(shape, generator=g, device=DEV) * 0.02
        return (w.to(torch.bfloat16), None) if c["wtype"] == "bf16" else _quantise(w, c["wtype"])

    c, op = case, case["op"]
    s = dict(case=case)
    if op == "linear_w4":
        w, ws = weights(c["N"], c["K"])
        s.update(x=rnd(c["T"], c["K"]), w=w, ws=ws, bias=rnd(c["N"], std=0.1) if c["bias"] else None,
                 residual=rnd(c["T"], c["N"]) if c["residual"] else None,
                 y=empty(c["T"], c["N"], dtype=torch.float32 if c["out"] == "fp32" else torch.bfloat16))
    elif op == "glu_w4":
        w, ws = weights(2 * c["I"], c["H"])
        s.update(x=rnd(c["T"], c["H"]), w=w, ws=ws, h=empty(c["T"], c["I"]))
    elif op == "rows":
        i32 = dict(dtype=torch.int32)
        s.update(ids=_routed(c["T"], c["E"], c["k"], c["skew"], g), offsets=empty(c["E"] + 1, **i32),
                 rows=empty(c["T"] * c["k"], **i32), places=empty(c["T"], c["k"], **i32))
    elif op in ("combine", "combine_backward"):
        T, k, H = c["T"], c["k"], c["H"]
        w = torch.rand((T, k), generator=g, device=DEV) + 0.05
        s.update(y=rnd(T * k, H), w=w / w.sum(1, keepdim=True),
                 places=torch.randperm(T * k, generator=g, device=DEV).to(torch.int32).view(T, k))
        if op == "combine":
            s.update(residual=rnd(T, H) if c["residual"] else None, out=empty(T, H))
        else:
            s.update(dout=rnd(T, H), dy=empty(T * k, H), dw=empty(T, k, dtype=torch.float32))
    else:
        T, E, k = c["T"], c["E"], c["k"]
        R = T * k
        offsets, rows, _ = _grouping(_routed(T, E, k, c["skew"], g), E)
        s.update(offsets=offsets, rows=rows, most=int((offsets[1:] - offsets[:-1]).max()))
        if op == "grouped_linear":
            w, ws = weights(E, c["N"], c["K"])
            s.update(x=rnd(R, c["K"]), w=w, ws=ws, bias=rnd(E, c["N"], std=0.1) if c["bias"] else None,
                     y=empty(R, c["N"]))
        elif op == "grouped_glu":
            w, ws = weights(E, 2 * c["I"], c["H"])
            s.update(x=rnd(T, c["H"]), w=w, ws=ws, h=empty(R, c["I"]), gu=empty(R, 2 * c["I"]) if c["save"] else None)
        else:
            H, I = c["H"], c["I"]
            s.update(dy=rnd(R, H), x=rnd(T, H), gu=rnd(R, 2 * I, std=0.02 * math.sqrt(H)), w13=rnd(E, 2 * I, H, std=0.02),
                     w2=rnd(E, H, I, std=0.02), dgu=empty(R, 2 * I), h=empty(R, I), dx=empty(R, H),
                     dw13=empty(E, 2 * I, H), dw2=empty(E, H, I))
    if c.get("wtype") == "mxfp4":
        s.update(table=torch.tensor(E2M1, device=DEV))
    return s


# ------------------------------------------------------------------ one pass

def run(s):
    return _own(s) if own else _plain(s)


def _own(s):
    import host_paged_expert_amd as pe
    c, op, stream = s["case"], s["case"]["op"], torch.cuda.current_stream()
    if op == "linear_w4":
        pe.linear_w4(s["x"], s["w"], s["ws"], s["y"], bias=s["bias"], act=c["act"], residual=s["residual"], stream=stream)
        return dict(y=s["y"])
    if op == "glu_w4":
        pe.glu_w4(s["x"], s["w"], s["ws"], s["h"], act=c["act"], stream=stream)
        return dict(h=s["h"])
    if op == "rows":
        pe.group_rows(s["ids"], s["offsets"], s["rows"], s["places"], stream=stream)
        return dict(offsets=s["offsets"], rows=s["rows"], places=s["places"])
    if op == "grouped_glu":
        pe.grouped_glu(s["x"], s["w"], s["h"], s["offsets"], rows=s["rows"], w_scales=s["ws"], act=c["act"], gu=s["gu"],
                       stream=stream)
        return dict(h=s["h"], gu=s["gu"])
    if op == "grouped_linear":
        pe.grouped_linear(s["x"], s["w"], s["y"], s["offsets"], w_scales=s["ws"], bias=s["bias"], stream=stream)
        return dict(y=s["y"])
    if op == "grouped_backward":
        pe.grouped_ffn_backward(s["dy"], s["x"], s["gu"], s["w13"], s["w2"], s["offsets"], s["dgu"], rows=s["rows"],
                                h=s["h"], dx=s["dx"], dw13=s["dw13"], dw2=s["dw2"], act=c["act"], stream=stream)
        return dict(dx=s["dx"], dw13=s["dw13"], dw2=s["dw2"])
    if op == "combine":
        pe.combine(s["y"], s["places"], s["out"], topk_w=s["w"], residual=s["residual"], stream=stream)
        return dict(out=s["out"])
    pe.combine_backward(s["dout"], s["places"], s["dy"], topk_w=s["w"], y=s["y"], dtopk_w=s["dw"], stream=stream)
    return dict(dy=s["dy"], dw=s["dw"])


def _act(v, act):
    if act == "silu":
        return v / (1 + torch.exp(-v))
    if act == "gelu":
        return 0.5 * v * (1 + torch.erf(v * math.sqrt(0.5)))
    return v


def _act_grad(v, act):
    if act == "silu":
        p = 1 / (1 + torch.exp(-v))
        return p * (1 + v * (1 - p))
    return 0.5 * (1 + torch.erf(v * math.sqrt(0.5))) + v * torch.exp(-0.5 * v * v) * (1 / math.sqrt(2 * math.pi))


def _weights32(s):
    w, ws = s["w"], s["ws"]
    if ws is None:
        return w.float()
    q = torch.stack((w & 15, w >> 4), -1).flatten(-2)
    if s["case"]["wtype"] == "int4":
        return (q.float() - 8) * ws.float().repeat_interleave(128, -1)
    return s["table"][q.int()] * torch.exp2(ws.float() - 127).repeat_interleave(32, -1)


def _slots(s, rows):
    """Every row's place in a [E, most, ...] array: its expert, and its place among that expert's rows."""
    p = torch.arange(rows, device=DEV)
    e = torch.searchsorted(s["offsets"], p, right=True, out_int32=True).long() - 1
    return e, p - s["offsets"][e]


def _spread(v, slot, s):
    """Rows in their experts' order as [E, most, columns], zeros behind each expert's last."""
    out = torch.zeros((s["offsets"].numel() - 1, s["most"], v.shape[1]), device=DEV)
    out[slot] = v.float()
    return out


def _plain(s):
    c, op, bf = s["case"], s["case"]["op"], torch.bfloat16
    if op == "linear_w4":
        y = s["x"].float() @ _weights32(s).t()
        if s["bias"] is not None:
            y = y + s["bias"].float()
        y = _act(y, c["act"])
        if s["residual"] is not None:
            y = y + s["residual"].float()
        return dict(y=y if c["out"] == "fp32" else y.to(bf))
    if op == "glu_w4":
        gu = s["x"].float() @ _weights32(s).t()
        return dict(h=(_act(gu[:, :c["I"]], c["act"]) * gu[:, c["I"]:]).to(bf))
    if op == "rows":
        offsets, rows, places = _grouping(s["ids"], c["E"])
        return dict(offsets=offsets, rows=rows, places=places)
    if op == "combine":
        y = (s["y"].float()[s["places"].long()] * s["w"][:, :, None]).sum(1)
        return dict(out=(y if s["residual"] is None else y + s["residual"].float()).to(bf))
    if op == "combine_backward":
        at, dout = s["places"].long(), s["dout"].float()
        dy = torch.empty_like(s["dy"])
        dy[at] = (s["w"][:, :, None] * dout[:, None, :]).to(bf)
        return dict(dy=dy, dw=(s["y"].float()[at] * dout[:, None, :]).sum(2))
    slot = _slots(s, c["T"] * c["k"])
    if op == "grouped_linear":
        y = torch.bmm(_spread(s["x"], slot, s), _weights32(s).transpose(1, 2).contiguous())[slot]
        return dict(y=(y if s["bias"] is None else y + s["bias"].float()[slot[0]]).to(bf))
    x = s["x"][s["rows"].long()]
    if op == "grouped_glu":
        gu = torch.bmm(_spread(x, slot, s), _weights32(s).transpose(1, 2).contiguous())[slot]
        h = _act(gu[:, :c["I"]], c["act"]) * gu[:, c["I"]:]
        return dict(h=h.to(bf), gu=gu.to(bf) if c["save"] else None)
    I = c["I"]
    g, u, dy = s["gu"][:, :I].float(), s["gu"][:, I:].float(), _spread(s["dy"], slot, s)
    dh = torch.bmm(dy, s["w2"].float())[slot]
    a = _act(g, c["act"])
    dgu = _spread(torch.cat((dh * u * _act_grad(g, c["act"]), dh * a), 1), slot, s)
    dx = torch.bmm(dgu, s["w13"].float())[slot]
    dw13 = torch.bmm(dgu.transpose(1, 2).contiguous(), _spread(x, slot, s))
    dw2 = torch.bmm(dy.transpose(1, 2).contiguous(), _spread(a * u, slot, s))
    return dict(dx=dx.to(bf), dw13=dw13.to(bf), dw2=dw2.to(bf))


# ------------------------------------------------------------------ bounds

def _experts(c):
    """Experts that T tokens of k distinct, equally likely ones reach, on average: the others' weights are not read."""
    return c["E"] * (1 - (1 - c["k"] / c["E"]) ** c["T"])


def work(case):
    c, op = case, case["op"]
    if op in ("linear_w4", "glu_w4"):
        T = c["T"]
        N, K = (c["N"], c["K"]) if op == "linear_w4" else (2 * c["I"], c["H"])
        w = N * K // 2 + (N * K // 64 if c["wtype"] == "int4" else N * K // 32)
        if op == "glu_w4":
            out = 2 * T * c["I"]
        else:
            out = (4 if c["out"] == "fp32" else 2) * T * N + (2 * N if c["bias"] else 0) + (2 * T * N if c["residual"] else 0)
        return {"bytes": w + 2 * T * K + out, "flops": 2 * T * N * K}
    if op == "rows":
        return {"bytes": 12 * c["T"] * c["k"] + 4 * (c["E"] + 1), "flops": 0}
    T, k = c["T"], c["k"]
    R = T * k
    if op == "combine":
        return {"bytes": 2 * R * c["H"] + 8 * R + (4 if c["residual"] else 2) * T * c["H"], "flops": 2 * R * c["H"]}
    if op == "combine_backward":
        return {"bytes": 4 * R * c["H"] + 2 * T * c["H"] + 12 * R, "flops": 3 * R * c["H"]}
    if op == "grouped_backward":
        H, I, e = c["H"], c["I"], _experts(c)
        # dy, x, gu and the reached experts' weights in; dx and every expert's gradients out; six products
        return {"bytes": int(2 * (2 * R * H + T * H + 2 * R * I + 3 * H * I * (e + c["E"]))) + 4 * R,
                "flops": 12 * R * H * I}
    N, K = (c["N"], c["K"]) if op == "grouped_linear" else (2 * c["I"], c["H"])
    each = {"bf16": 2.0, "int4": 0.5 + 1 / 64, "mxfp4": 0.5 + 1 / 32}[c["wtype"]]
    out = 2 * R * N + (2 * int(_experts(c)) * N if c["bias"] else 0) if op == "grouped_linear" else \
        2 * R * c["I"] + (4 * R * c["I"] if c["save"] else 0)
    rows = R if op == "grouped_linear" else T
    return {"bytes": int(_experts(c) * N * K * each) + 2 * rows * K + out + 4 * R, "flops": 2 * R * N * K}


# ------------------------------------------------------------------ 64 bits

def _decoded64(codes, scales, wtype):
    """Weights in 64 bits, the last dimension restored from its packed codes."""
    if scales is None:
        return codes.double()
    low = torch.bitwise_and(codes.int(), 15)
    high = torch.bitwise_right_shift(codes.int(), 4)
    q = torch.empty((*codes.shape[:-1], 2 * codes.shape[-1]), dtype=torch.int32, device=codes.device)
    q[..., 0::2], q[..., 1::2] = low, high
    if wtype == "int4":
        per = scales.double()
        value = (q - 8).double()
    else:
        per = torch.pow(torch.tensor(2.0, dtype=torch.float64, device=codes.device), scales.double() - 127)
        exponent, mantissa = (q >> 1) & 3, (q & 1).double()
        size = torch.where(exponent == 0, 0.5 * mantissa, (1 + 0.5 * mantissa) * torch.exp2((exponent - 1).double()))
        value = torch.where(q >= 8, -size, size)
    each = value.shape[-1] // per.shape[-1]
    return (value.view(*per.shape, each) * per[..., None]).reshape(value.shape)


def _cdf64(v):
    return 0.5 * torch.special.erfc(-v / math.sqrt(2.0))


def _act64(v, act):
    return v * torch.sigmoid(v) if act == "silu" else v * _cdf64(v) if act == "gelu" else v


def exact(case, seed):
    s = prepare(case, seed)
    c, op = case, case["op"]
    if op == "rows":
        ids = s["ids"].cpu().reshape(-1).tolist()
        groups = [[] for _ in range(c["E"])]
        for i, e in enumerate(ids):
            groups[e].append(i)
        offsets, rows, places = [0], [], [0] * len(ids)
        for members in groups:
            for i in members:
                places[i] = len(rows)
                rows.append(i // c["k"])
            offsets.append(len(rows))
        i32 = dict(dtype=torch.int32)
        return dict(offsets=torch.tensor(offsets, **i32), rows=torch.tensor(rows, **i32),
                    places=torch.tensor(places, **i32).view(c["T"], c["k"]))
    if op in ("combine", "combine_backward"):
        w, y, at = s["w"].double(), s["y"].double(), s["places"].long()
        if op == "combine":
            out = s["residual"].double() if c["residual"] else torch.zeros((c["T"], c["H"]), dtype=torch.float64, device=DEV)
            for j in range(c["k"]):
                out = out + w[:, j:j + 1] * y[at[:, j]]
            return dict(out=out)
        dout, dy, dw = s["dout"].double(), torch.zeros_like(y), torch.zeros_like(w)
        for j in range(c["k"]):
            dy[at[:, j]] = w[:, j:j + 1] * dout
            dw[:, j] = (dout * y[at[:, j]]).sum(1)
        return dict(dy=dy, dw=dw)
    if op in ("linear_w4", "glu_w4"):
        y = torch.mm(s["x"].double(), _decoded64(s["w"], s["ws"], c["wtype"]).T.contiguous())
        if op == "glu_w4":
            gate, up = y.split(c["I"], 1)
            return dict(h=_act64(gate, c["act"]) * up)
        y = _act64(y + s["bias"].double() if c["bias"] else y, c["act"])
        return dict(y=y + s["residual"].double() if c["residual"] else y)

    bounds = s["offsets"].tolist()
    token = s["rows"].long()

    def rows(e):
        return slice(bounds[e], bounds[e + 1])

    if op in ("grouped_linear", "grouped_glu"):
        N = c["N"] if op == "grouped_linear" else 2 * c["I"]
        y = torch.empty((c["T"] * c["k"], N), dtype=torch.float64, device=DEV)
        for e in range(c["E"]):
            x = s["x"][rows(e)] if op == "grouped_linear" else s["x"][token[rows(e)]]
            w = _decoded64(s["w"][e], None if s["ws"] is None else s["ws"][e], c["wtype"])
            y[rows(e)] = torch.mm(x.double(), w.T.contiguous())
            if op == "grouped_linear" and c["bias"]:
                y[rows(e)] += s["bias"][e].double()
        if op == "grouped_linear":
            return dict(y=y)
        gate, up = y.split(c["I"], 1)
        return dict(h=_act64(gate, c["act"]) * up, gu=y if c["save"] else None)
    I, H = c["I"], c["H"]
    f64 = dict(dtype=torch.float64, device=DEV)
    dx, dw13, dw2 = torch.empty((c["T"] * c["k"], H), **f64), torch.empty((c["E"], 2 * I, H), **f64), torch.empty((c["E"], H, I), **f64)
    for e in range(c["E"]):
        r = rows(e)
        gate, up = s["gu"][r].double().split(I, 1)
        dy, x, w13, w2 = s["dy"][r].double(), s["x"][token[r]].double(), s["w13"][e].double(), s["w2"][e].double()
        if c["act"] == "silu":
            sig = torch.sigmoid(gate)
            slope = sig + gate * sig * (1 - sig)
        else:
            slope = _cdf64(gate) + gate * torch.exp(-gate.square() / 2) / math.sqrt(2 * math.pi)
        dh, act = torch.mm(dy, w2), _act64(gate, c["act"])
        both = torch.cat((dh * up * slope, dh * act), 1)
        dx[r] = torch.mm(both, w13)
        dw13[e] = torch.mm(both.T.contiguous(), x)
        dw2[e] = torch.mm(dy.T.contiguous(), act * up)
    return dict(dx=dx, dw13=dw13, dw2=dw2)
