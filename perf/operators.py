"""Timed cases of the dense operators around a paged MoE layer.

An MoE block calls them in this order: `rmsnorm` (the residual's addition, the
norm, and an e4m3 output with scales where the projections after it are FP8),
`linear` (the router's logits), `route` (top-k ids and weights for pe_forward),
`glu` (gate and up projection, activation and product of the always-on shared
expert or of a dense layer), `linear` again (its down projection with the
residual in the epilogue), and `ffn_backward` (the gradients of that
feed-forward block).

`own` chooses between plain torch arithmetic in 32 bits and libpe's kernels.
Sizes: hidden 2048 and expert intermediate 768 with 128 experts, top-8, and
hidden 2880 with 32 experts, top-4, are the workloads of synth/workloads.py;
an intermediate of 6144 is as wide as eight experts of 768 together; 2048
tokens is the prefill chunk.
"""
import math

import torch

own = False

DEV = "cuda"
E4M3_MAX = 448.0
TINY = 2.0 ** -126


# ------------------------------------------------------------------ cases

def listed():
    return [
        # The norm before the MoE of a decode step of four requests; its output feeds FP8 projections.
        dict(name="norm_decode_fp8", op="norm", T=4, H=2048, out="fp8", residual=True),
        # The same norm over a long prefill at the widest hidden size the paged layer takes.
        dict(name="norm_prefill_bf16", op="norm", T=8192, H=4096, out="bf16", residual=True),
        # Top-8 of 128 experts for a decode step of four requests.
        dict(name="route_decode", op="route", T=4, E=128, k=8, scoring="softmax", renorm=True),
        # The same choice for a long prefill.
        dict(name="route_prefill", op="route", T=8192, E=128, k=8, scoring="softmax", renorm=True),
        # Router logits of a decode step, kept in fp32 for the choice of experts.
        dict(name="router_logits_decode", op="linear", wtype="bf16", T=4, N=128, K=2048, bias=True, act="none",
             residual=False, out="fp32"),
        # A square projection with bias and residual, hidden 2880, over an odd number of tokens.
        dict(name="linear_bf16_odd", op="linear", wtype="bf16", T=1023, N=2880, K=2880, bias=True, act="none",
             residual=True, out="bf16"),
        # Down projection of the dense block over a prefill chunk, FP8, added to the residual stream.
        dict(name="linear_down_fp8", op="linear", wtype="fp8", T=2048, N=2048, K=6144, bias=False, act="none",
             residual=True, out="bf16"),
        # One decode token through the dense block's gate/up half: bound by the weights' bytes.
        dict(name="glu_decode_bf16", op="glu", wtype="bf16", T=1, H=2048, I=6144, act="silu", save=False),
        # A prefill chunk through it, keeping what the backward pass needs.
        dict(name="glu_prefill_bf16", op="glu", wtype="bf16", T=2048, H=2048, I=6144, act="silu", save=True),
        # A prefill chunk through it in FP8, output ready for the FP8 down projection.
        dict(name="glu_prefill_fp8", op="glu", wtype="fp8", T=2048, H=2048, I=6144, act="silu", save=False),
        # Gradients of a shared expert of one routed expert's size over a short, odd batch.
        dict(name="ffn_backward_small", op="ffn_backward", T=257, H=2048, I=768, act="silu"),
        # Gradients of the dense block over two prefill chunks.
        dict(name="ffn_backward_large", op="ffn_backward", T=4096, H=2048, I=6144, act="silu"),
    ]


def _log(rng, lo, hi, step=1):
    """An integer in [lo, hi], spread over its logarithm, a multiple of `step`."""
    v = math.exp(rng.uniform(math.log(lo), math.log(hi + 0.999)))
    return max(lo, min(hi, int(v) // step * step))


def draw(rng):
    op = rng.choice(["norm", "route", "linear", "glu", "ffn_backward"])
    if op == "norm":
        out = rng.choice(["bf16", "fp8"])
        return dict(op=op, T=_log(rng, 1, 8192), H=_log(rng, 128, 4096, 128 if out == "fp8" else 8), out=out,
                    residual=rng.random() < 0.7)
    if op == "route":
        E = _log(rng, 8, 256)
        return dict(op=op, T=_log(rng, 1, 8192), E=E, k=rng.randint(1, min(E, 10)),
                    scoring=rng.choice(["softmax", "sigmoid"]), renorm=rng.random() < 0.7)
    wtype = rng.choice(["bf16", "fp8"])
    step = 128 if wtype == "fp8" else 8
    if op == "linear":
        return dict(op=op, wtype=wtype, T=_log(rng, 1, 4096), N=_log(rng, 16, 6144), K=_log(rng, 128, 6144, step),
                    bias=rng.random() < 0.5, act=rng.choice(["none", "silu", "gelu"]), residual=rng.random() < 0.5,
                    out="bf16" if wtype == "fp8" else rng.choice(["bf16", "fp32"]))
    act = rng.choice(["silu", "gelu"])
    if op == "glu":
        return dict(op=op, wtype=wtype, T=_log(rng, 1, 4096), H=_log(rng, 128, 4096, step),
                    I=_log(rng, 128, 6144, step), act=act, save=wtype == "bf16" and rng.random() < 0.5)
    return dict(op=op, T=_log(rng, 1, 4096), H=_log(rng, 128, 2048, 8), I=_log(rng, 128, 6144, 8), act=act)


# ------------------------------------------------------------------ inputs

def _to_fp8_rows(v):
    """e4m3 codes and fp32 scales per row and 128 columns, as the norm gives them."""
    T, C = v.shape
    g = v.float().view(T, C // 128, 128)
    s = (g.abs().amax(2) / E4M3_MAX).clamp_min(TINY)
    return (g / s[:, :, None]).clamp(-E4M3_MAX, E4M3_MAX).view(T, C).to(torch.float8_e4m3fn), s


def _to_fp8_blocks(w):
    """e4m3 codes and one fp32 scale per 128x128 block (the last block row may be short)."""
    N, K = w.shape
    nb = -(-N // 128)
    p = torch.zeros((nb * 128, K), device=w.device)
    p[:N] = w.float()
    b = p.view(nb, 128, K // 128, 128)
    s = (b.abs().amax((1, 3)) / E4M3_MAX).clamp_min(TINY)
    q = (b / s[:, None, :, None]).clamp(-E4M3_MAX, E4M3_MAX).view(nb * 128, K)[:N].to(torch.float8_e4m3fn)
    return q.contiguous(), s.contiguous()


def prepare(case, seed):
    g = torch.Generator(device=DEV).manual_seed(seed)

    def rnd(*shape, std=1.0, dtype=torch.bfloat16):
        return (torch.randn(shape, generator=g, device=DEV) * std).to(dtype)

    def empty(*shape, dtype=torch.bfloat16):
        return torch.empty(shape, dtype=dtype, device=DEV)

    c, op = case, case["op"]
    s = dict(case=case)
    if op == "norm":
        T, H = c["T"], c["H"]
        s.update(x=rnd(T, H), residual=rnd(T, H) if c["residual"] else None,
                 weight=(1 + 0.1 * torch.randn(H, generator=g, device=DEV)).to(torch.bfloat16),
                 sum=empty(T, H) if c["residual"] else None)
        if c["out"] == "fp8":
            s.update(y=empty(T, H, dtype=torch.float8_e4m3fn), scales=empty(T, H // 128, dtype=torch.float32))
        else:
            s.update(y=empty(T, H), scales=None)
    elif op == "route":
        T, E, k = c["T"], c["E"], c["k"]
        s.update(logits=rnd(T, E, std=2.0, dtype=torch.float32), ids=empty(T, k, dtype=torch.int32),
                 weights=empty(T, k, dtype=torch.float32))
    elif op == "linear":
        T, N, K = c["T"], c["N"], c["K"]
        x, w, xs, ws = rnd(T, K), rnd(N, K, std=0.02), None, None
        if c["wtype"] == "fp8":
            (x, xs), (w, ws) = _to_fp8_rows(x), _to_fp8_blocks(w)
        s.update(x=x, w=w, xs=xs, ws=ws, bias=rnd(N, std=0.1) if c["bias"] else None,
                 residual=rnd(T, N) if c["residual"] else None,
                 y=empty(T, N, dtype=torch.float32 if c["out"] == "fp32" else torch.bfloat16))
    elif op == "glu":
        T, H, I = c["T"], c["H"], c["I"]
        x, w, xs, ws = rnd(T, H), rnd(2 * I, H, std=0.02), None, None
        if c["wtype"] == "fp8":
            (x, xs), (w, ws) = _to_fp8_rows(x), _to_fp8_blocks(w)
            s.update(h=empty(T, I, dtype=torch.float8_e4m3fn), hs=empty(T, I // 128, dtype=torch.float32))
        else:
            s.update(h=empty(T, I), hs=None)
        s.update(x=x, w=w, xs=xs, ws=ws, gu=empty(T, 2 * I) if c["save"] else None)
    else:
        T, H, I = c["T"], c["H"], c["I"]
        x, w13 = rnd(T, H), rnd(2 * I, H, std=0.02)
        s.update(x=x, w13=w13, w2=rnd(H, I, std=0.02), gu=(x.float() @ w13.float().t()).to(torch.bfloat16),
                 dy=rnd(T, H), dgu=empty(T, 2 * I), h=empty(T, I), dx=empty(T, H), dw13=empty(2 * I, H),
                 dw2=empty(H, I))
    return s


# ------------------------------------------------------------------ one pass

def run(s):
    return _own(s) if own else _plain(s)


def _own(s):
    import host_paged_expert_amd as pe
    c, op, stream = s["case"], s["case"]["op"], torch.cuda.current_stream()
    if op == "norm":
        pe.rmsnorm(s["x"], s["weight"], 1e-6, s["y"], scales=s["scales"], residual=s["residual"], sum_out=s["sum"],
                   stream=stream)
        return dict(y=s["y"], scales=s["scales"], sum=s["sum"])
    if op == "route":
        pe.route(s["logits"], s["ids"], s["weights"], scoring=c["scoring"], renormalize=c["renorm"], stream=stream)
        return dict(ids=s["ids"], weights=s["weights"])
    if op == "linear":
        pe.linear(s["x"], s["w"], s["y"], x_scales=s["xs"], w_scales=s["ws"], bias=s["bias"], act=c["act"],
                  residual=s["residual"], stream=stream)
        return dict(y=s["y"])
    if op == "glu":
        pe.glu(s["x"], s["w"], s["h"], x_scales=s["xs"], w_scales=s["ws"], out_scales=s["hs"], act=c["act"],
               gu=s["gu"], stream=stream)
        return dict(h=s["h"], scales=s["hs"], gu=s["gu"])
    pe.ffn_backward(s["dy"], s["x"], s["gu"], s["w13"], s["w2"], s["dgu"], s["h"], dx=s["dx"], dw13=s["dw13"],
                    dw2=s["dw2"], act=c["act"], stream=stream)
    return dict(dx=s["dx"], dw13=s["dw13"], dw2=s["dw2"])


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


def _rows32(x, xs):
    x = x.float()
    return x if xs is None else x * xs.repeat_interleave(128, 1)


def _weights32(w, ws):
    w = w.float()
    return w if ws is None else w * ws.repeat_interleave(128, 0)[:w.shape[0]].repeat_interleave(128, 1)


def _plain(s):
    c, op = s["case"], s["case"]["op"]
    if op == "norm":
        v = s["x"].float()
        if s["residual"] is not None:
            v = v + s["residual"].float()
        y = v * (1 / torch.sqrt((v * v).mean(1, keepdim=True) + 1e-6)) * s["weight"].float()
        total = v.to(torch.bfloat16) if s["residual"] is not None else None
        if c["out"] == "bf16":
            return dict(y=y.to(torch.bfloat16), scales=None, sum=total)
        codes, scales = _to_fp8_rows(y)
        return dict(y=codes, scales=scales, sum=total)
    if op == "route":
        top, ids = torch.sort(s["logits"], dim=1, descending=True, stable=True)
        if c["scoring"] == "softmax":
            e = torch.exp(top - top[:, :1])
            p = (e / e.sum(1, keepdim=True))[:, :c["k"]]
        else:
            p = 1 / (1 + torch.exp(-top[:, :c["k"]]))
        if c["renorm"]:
            p = p / p.sum(1, keepdim=True)
        return dict(ids=ids[:, :c["k"]].to(torch.int32), weights=p.contiguous())
    if op == "linear":
        y = _rows32(s["x"], s["xs"]) @ _weights32(s["w"], s["ws"]).t()
        if s["bias"] is not None:
            y = y + s["bias"].float()
        y = _act(y, c["act"])
        if s["residual"] is not None:
            y = y + s["residual"].float()
        return dict(y=y if c["out"] == "fp32" else y.to(torch.bfloat16))
    if op == "glu":
        gu = _rows32(s["x"], s["xs"]) @ _weights32(s["w"], s["ws"]).t()
        h = _act(gu[:, :c["I"]], c["act"]) * gu[:, c["I"]:]
        if c["wtype"] == "fp8":
            codes, scales = _to_fp8_rows(h)
            return dict(h=codes, scales=scales, gu=None)
        return dict(h=h.to(torch.bfloat16), scales=None, gu=gu.to(torch.bfloat16) if c["save"] else None)
    I = c["I"]
    x, dy, g, u = s["x"].float(), s["dy"].float(), s["gu"][:, :I].float(), s["gu"][:, I:].float()
    dh = dy @ s["w2"].float()
    a = _act(g, c["act"])
    dgu = torch.cat((dh * u * _act_grad(g, c["act"]), dh * a), 1)
    bf = torch.bfloat16
    return dict(dx=(dgu @ s["w13"].float()).to(bf), dw13=(dgu.t() @ x).to(bf), dw2=(dy.t() @ (a * u)).to(bf))


# ------------------------------------------------------------------ bounds

def work(case):
    c, op = case, case["op"]
    if op == "norm":
        n = c["T"] * c["H"]
        out = n + 4 * (n // 128) if c["out"] == "fp8" else 2 * n
        return {"bytes": 2 * n + (4 * n if c["residual"] else 0) + 2 * c["H"] + out, "flops": 5 * n}
    if op == "route":
        n = c["T"] * c["E"]
        return {"bytes": 4 * n + 8 * c["T"] * c["k"], "flops": 4 * n}
    if op == "linear":
        T, N, K = c["T"], c["N"], c["K"]
        b = 1 if c["wtype"] == "fp8" else 2
        scales = 4 * (T * K // 128 + -(-N // 128) * (K // 128)) if b == 1 else 0
        return {"bytes": b * (T * K + N * K) + scales + (2 * N if c["bias"] else 0) +
                (2 * T * N if c["residual"] else 0) + (4 if c["out"] == "fp32" else 2) * T * N,
                "flops": 2 * T * N * K}
    T, H, I = c["T"], c["H"], c["I"]
    if op == "glu":
        b = 1 if c["wtype"] == "fp8" else 2
        scales = 4 * (T * H // 128 + (2 * I // 128) * (H // 128) + T * I // 128) if b == 1 else 0
        return {"bytes": b * (T * H + 2 * I * H + T * I) + scales + (4 * T * I if c["save"] else 0),
                "flops": 4 * T * H * I}
    # dy, x, gu, w13 and w2 in; dx, dw13 and dw2 out; six products of T x H x I
    return {"bytes": 2 * (3 * T * H + 2 * T * I + 2 * 3 * H * I), "flops": 12 * T * H * I}


# ------------------------------------------------------------------ 64 bits

def _e4m3_grid(v):
    """The e4m3 value nearest each v (ties to the even code), largest 448, in 64 bits."""
    a = v.abs().clamp(max=E4M3_MAX)
    step = torch.exp2(torch.floor(torch.log2(a.clamp_min(2.0 ** -6))) - 3)
    return torch.sign(v) * (torch.round(a / step) * step).clamp(max=E4M3_MAX)


def _quantised64(v):
    T, C = v.shape
    blocks = v.reshape(T, C // 128, 128)
    scale = torch.clamp(blocks.abs().max(2).values / E4M3_MAX, min=TINY)
    return _e4m3_grid(blocks / scale.unsqueeze(2)).reshape(T, C), scale


def _normal_cdf64(v):
    return 0.5 * torch.special.erfc(-v / math.sqrt(2.0))


def exact(case, seed):
    s = prepare(case, seed)
    c, op, f64 = case, case["op"], torch.float64

    def wide(codes, scales):
        """Values of a matrix: scales cover 128 columns, and one row or 128 rows."""
        m = codes.to(f64)
        if scales is None:
            return m
        rows = torch.arange(m.shape[0], device=DEV)
        if scales.shape[0] != m.shape[0] or codes is s.get("w"):
            rows = rows // 128
        cols = torch.arange(m.shape[1], device=DEV) // 128
        return m * scales.to(f64)[rows][:, cols]

    def activation(v):
        return v * torch.sigmoid(v) if c["act"] == "silu" else v * _normal_cdf64(v) if c["act"] == "gelu" else v

    if op == "norm":
        v = s["x"].to(f64) + (s["residual"].to(f64) if c["residual"] else 0)
        y = s["weight"].to(f64) * v / torch.sqrt(v.square().sum(1, keepdim=True) / c["H"] + 1e-6)
        total = v if c["residual"] else None
        if c["out"] == "bf16":
            return dict(y=y, scales=None, sum=total)
        codes, scales = _quantised64(y)
        return dict(y=codes, scales=scales, sum=total)
    if op == "route":
        lg = s["logits"].to(f64)
        p = torch.softmax(lg, 1) if c["scoring"] == "softmax" else torch.sigmoid(lg)
        ids = torch.argsort(-lg, dim=1, stable=True)[:, :c["k"]]
        w = torch.gather(p, 1, ids)
        return dict(ids=ids.to(torch.int32), weights=w / w.sum(1, keepdim=True) if c["renorm"] else w)
    if op == "linear":
        y = torch.mm(wide(s["x"], s["xs"]), wide(s["w"], s["ws"]).T.contiguous())
        y = activation(y + s["bias"].to(f64) if c["bias"] else y)
        return dict(y=y + s["residual"].to(f64) if c["residual"] else y)
    if op == "glu":
        both = torch.mm(wide(s["x"], s["xs"]), wide(s["w"], s["ws"]).T.contiguous())
        gate, up = both.split(c["I"], 1)
        h = activation(gate) * up
        if c["wtype"] == "fp8":
            codes, scales = _quantised64(h)
            return dict(h=codes, scales=scales, gu=None)
        return dict(h=h, scales=None, gu=both if c["save"] else None)
    gate, up = (t.to(f64) for t in s["gu"].split(c["I"], 1))
    x, dy, w13, w2 = (s[n].to(f64) for n in ("x", "dy", "w13", "w2"))
    dh = torch.mm(dy, w2)
    if c["act"] == "silu":
        sig = torch.sigmoid(gate)
        slope = sig + gate * sig * (1 - sig)
    else:
        slope = _normal_cdf64(gate) + gate * torch.exp(-gate.square() / 2) / math.sqrt(2 * math.pi)
    act = activation(gate)
    dgate, dup = dh * up * slope, dh * act
    return dict(dx=torch.mm(dgate, w13[:c["I"]]) + torch.mm(dup, w13[c["I"]:]),
                dw13=torch.cat((torch.mm(dgate.T.contiguous(), x), torch.mm(dup.T.contiguous(), x))),
                dw2=torch.mm(dy.T.contiguous(), act * up))
