"""What is measured of the routed experts' training operators and of their 16-bit products.

Four operators, each in its directions and types:

  product   out[r] = a[r] @ W[e(r)]^T, rows grouped by expert (ragged), 16-bit operands.  "forward" takes
            W [E, N, K]; "data_grad" takes W [E, K, N] as the forward holds it and reduces over its rows;
            "slot" is the decode form: each route names its expert's slot, a negative slot gives a zero row.
  wgrad     dW[e] = dy[rows of e]^T @ a[rows of e]; `a` in 16 bits, or saved in 8 bits (e4m3 codes with one
            power-of-two scale per 1 x 128 group).
  saved     activations saved in 8 bits for the backward pass: "save" forms act(gate) * up and the codes and
            scales of [gate | up] ("save_rows": of plain rows); "use" is the activation's backward from them.
  combine   the backward of the routing-weighted sum over a token's routes, through to the router's logits.
"""
import math

import numpy as np
import torch

own = False

DT = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
ACTS = {"silu": 1, "gelu": 2, "relu": 3, "sigmoid": 4, "mul": 5}


# ---------------------------------------------------------------- the cases

def listed():
    return [
        # one token's eight routes against a pool of 64 resident experts, one route inactive: a decode step's gate/up
        dict(name="slot_decode_gate_up", op="product", form="slot", dt="bf16", out="fp32", experts=64, rows=8,
             per_token=8, off=1, n=1536, k=2048),
        # a prefill of 4096 tokens over 256 experts, six each: about 96 rows an expert, the weights dominate
        dict(name="forward_gate_up_e256", op="product", form="forward", dt="bf16", out="bf16", experts=256,
             rows=24576, skew=0.0, n=2048, k=4096),
        # few large experts in training: the gradient of the layer's input through gate/up
        dict(name="data_grad_gate_up_e8", op="product", form="data_grad", dt="bf16", out="bf16", experts=8,
             rows=16384, skew=0.1, n=4096, k=8192),
        # a short ragged batch with widths that fit no tile, some experts empty
        dict(name="forward_ragged_odd", op="product", form="forward", dt="fp16", out="fp16", experts=16,
             rows=333, skew=1.5, n=1000, k=520),
        # few large experts in training: fp32 gradients of gate/up
        dict(name="wgrad_gate_up_e8", op="wgrad", saved=False, dt="bf16", out="fp32", experts=8, rows=16384,
             skew=0.1, n=8192, k=4096),
        # many experts with few rows each, the layer's input kept in 8 bits: the gradients' bytes dominate
        dict(name="wgrad_saved_e256", op="wgrad", saved=True, dt="bf16", out="bf16", experts=256, rows=24576,
             skew=0.0, n=2048, k=4096),
        # small experts and long row ranges: few output tiles, a long reduction
        dict(name="wgrad_long_rows", op="wgrad", saved=False, dt="fp16", out="fp32", experts=4, rows=20001,
             skew=0.5, n=512, k=768),
        # the forward's activation of a 24576-route step, [gate | up] saved for the backward pass
        dict(name="save_gate_up", op="saved", form="save", act="silu", dt="bf16", rows=24576, n=1024),
        # its backward
        dict(name="use_gate_up", op="saved", form="use", act="silu", dt="bf16", rows=24576, n=1024),
        # a few rows of a small layer with a width that ends inside a group
        dict(name="use_small_odd", op="saved", form="use", act="gelu", dt="fp16", rows=37, n=712),
        # 4096 tokens, six routes each, rows in expert order
        dict(name="combine_prefill", op="combine", dt="bf16", tokens=4096, topk=6, h=4096, experts=256, off=0.0,
             mapped=True),
        # a few tokens in route order with dropped routes
        dict(name="combine_small", op="combine", dt="fp32", tokens=9, topk=8, h=2048, experts=64, off=0.2,
             mapped=False),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _log8(rng, lo, hi):
    return 8 * max(1, _log(rng, lo / 8, hi / 8))


def draw(rng):
    while True:
        op = rng.choice(["product", "product", "product", "wgrad", "wgrad", "saved", "saved", "combine"])
        if op == "product":
            form = rng.choice(["forward", "data_grad", "slot"])
            c = dict(op=op, form=form, dt=rng.choice(["bf16", "fp16"]), out=rng.choice(["bf16", "fp16", "fp32"]),
                     n=_log8(rng, 64, 8192), k=_log8(rng, 64, 8192))
            if form == "slot":
                per = rng.choice([1, 2, 6, 8])
                c.update(experts=_log(rng, 1, 64), rows=per * _log(rng, 1, 8), per_token=per, off=rng.choice([0, 1]))
            else:
                c.update(experts=_log(rng, 1, 256), rows=_log(rng, 1, 24576), skew=rng.uniform(0.0, 1.0))
        elif op == "wgrad":
            saved = rng.random() < 0.5
            c = dict(op=op, saved=saved, dt=rng.choice(["bf16", "fp16"]), out=rng.choice(["bf16", "fp16", "fp32"]),
                     experts=_log(rng, 1, 256), rows=_log(rng, 1, 24576), skew=rng.uniform(0.0, 1.0),
                     n=_log8(rng, 64, 8192), k=_log8(rng, 64, 8192))
            if saved:
                c["k"] = 16 * ((c["k"] + 8) // 16)
        elif op == "saved":
            c = dict(op=op, form=rng.choice(["save", "save_rows", "use", "use"]), act=rng.choice(sorted(ACTS)),
                     dt=rng.choice(["bf16", "fp16"]), rows=_log(rng, 1, 24576), n=_log8(rng, 64, 4096))
        else:
            experts = _log(rng, 8, 512)
            c = dict(op=op, dt=rng.choice(["bf16", "fp16", "fp32"]), tokens=_log(rng, 1, 4096),
                     topk=rng.randint(1, 8), h=_log8(rng, 64, 8192), experts=experts,
                     off=rng.choice([0.0, 0.1, 0.5]), mapped=rng.random() < 0.5)
        w = work(c)
        if w["flops"] <= 1.1e12 and w["bytes"] <= 4.4e9 and (op == "product" or op == "wgrad" or w["bytes"] <= 6.2e8):
            return c


def work(case):
    c = case
    if c["op"] == "product":
        R, E, n, k = c["rows"], c["experts"], c["n"], c["k"]
        if c["form"] == "slot":
            R = R - c["off"]
            a = -(-c["rows"] // c["per_token"]) * k * 2
        else:
            a = R * k * 2
        used = E * (1.0 - (1.0 - 1.0 / E) ** R)          # experts that some row names
        size = 4 if c["out"] == "fp32" else 2
        return dict(bytes=int(a + used * n * k * 2 + c["rows"] * n * size), flops=2 * R * n * k)
    if c["op"] == "wgrad":
        R, E, n, k = c["rows"], c["experts"], c["n"], c["k"]
        a = R * (k + 4 * -(-k // 128)) if c["saved"] else R * k * 2
        size = 4 if c["out"] == "fp32" else 2
        return dict(bytes=R * n * 2 + a + E * n * k * size, flops=2 * R * n * k)
    if c["op"] == "saved":
        R, n, g = c["rows"], c["n"], 4 * -(-c["n"] // 128)
        if c["form"] == "save":
            return dict(bytes=R * (4 * n + 2 * n + 2 * n + 2 * g), flops=20 * R * n)
        if c["form"] == "save_rows":
            return dict(bytes=R * (2 * n + n + g), flops=5 * R * n)
        return dict(bytes=R * (2 * n + 2 * n + 2 * g + 4 * n + 2 * n), flops=25 * R * n)
    T, R, h = c["tokens"], c["tokens"] * c["topk"], c["h"]
    size = 4 if c["dt"] == "fp32" else 2
    return dict(bytes=T * h * 2 + 2 * R * h * size + 4 * T * c["experts"] + 24 * R, flops=4 * R * h)


# --------------------------------------------------------------- the inputs

def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed & 0x7FFFFFFFFFFF)
    return g


def _randn(g, shape, std, dt):
    """Normal values of type dt, drawn in pieces so that a large bank needs no 32-bit copy of itself."""
    out = torch.empty(shape, dtype=dt, device="cuda")
    flat = out.view(-1)
    for i in range(0, flat.numel(), 1 << 28):
        part = flat[i:i + (1 << 28)]
        part.copy_(torch.randn(part.numel(), generator=g, device="cuda", dtype=torch.float32) * std)
    return out


def _counts(c, seed):
    """Rows of each expert: multinomial over popularities e^(skew z), as a router with hot and cold experts gives."""
    rng = np.random.default_rng(seed)
    p = np.exp(c["skew"] * rng.standard_normal(c["experts"]))
    return rng.multinomial(c["rows"], p / p.sum())


def _groups(counts):
    """The device plan of rows grouped by expert: offsets, and the places of a padded [E, longest] form."""
    offs = np.concatenate([[0], np.cumsum(counts)]).astype(np.int32)
    cap = max(1, int(counts.max()))
    expert = np.repeat(np.arange(len(counts)), counts)
    place = np.arange(int(counts.sum())) - offs[:-1][expert]
    pad = np.minimum(offs[:-1, None] + np.arange(cap)[None, :], max(0, int(counts.sum()) - 1))
    there = np.arange(cap)[None, :] < counts[:, None]
    dev = lambda x: torch.from_numpy(np.ascontiguousarray(x)).cuda()  # noqa: E731
    return dict(offsets=dev(offs), expert=dev(expert.astype(np.int64)), place=dev(place.astype(np.int64)),
                pad=dev(pad.astype(np.int64)), there=dev(there))


def _quantised(x):
    """e4m3 codes and power-of-two scales of 1 x 128 groups, as a forward pass saves them."""
    q, s = _save_plain(x.float())
    return q.view(torch.uint8), s


def _inputs(case, seed):
    c, g = case, _gen(seed)
    if c["op"] == "product":
        dt = DT[c["dt"]]
        if c["form"] == "slot":
            rng = np.random.default_rng(seed)
            slots = rng.integers(0, c["experts"], size=c["rows"]).astype(np.int32)
            if c["off"] and c["rows"] > 1:
                slots[rng.integers(0, c["rows"])] = -1
            tokens = -(-c["rows"] // c["per_token"])
            return dict(a=_randn(g, (tokens, c["k"]), 1.0, dt), w=_randn(g, (c["experts"], c["n"], c["k"]), 0.02, dt),
                        slots=torch.from_numpy(slots).cuda())
        counts = _counts(c, seed)
        shape = (c["experts"], c["n"], c["k"]) if c["form"] == "forward" else (c["experts"], c["k"], c["n"])
        std = 1.0 if c["form"] == "forward" else 0.05
        return dict(a=_randn(g, (c["rows"], c["k"]), std, dt), w=_randn(g, shape, 0.02, dt), counts=counts,
                    **_groups(counts))
    if c["op"] == "wgrad":
        counts = _counts(c, seed)
        d = dict(dy=_randn(g, (c["rows"], c["n"]), 0.05, DT[c["dt"]]), counts=counts, **_groups(counts))
        a = _randn(g, (c["rows"], c["k"]), 1.0, DT[c["dt"]])
        if c["saved"]:
            d["a"], d["a_s"] = _quantised(a)
        else:
            d["a"], d["a_s"] = a, None
        return d
    if c["op"] == "saved":
        dt, R, n = DT[c["dt"]], c["rows"], c["n"]
        if c["form"] == "save_rows":
            return dict(x=_randn(g, (R, n), 1.0, dt))
        x = _randn(g, (R, 2 * n), 1.3, dt)
        if c["form"] == "save":
            return dict(x=x)
        (qg, sg), (qu, su) = _quantised(x[:, :n]), _quantised(x[:, n:])
        return dict(dh=_randn(g, (R, n), 0.05, dt), q=torch.cat([qg, qu], 1), s=torch.cat([sg, su], 1))
    T, k, h, E = c["tokens"], min(c["topk"], c["experts"]), c["h"], c["experts"]
    logits = torch.randn((T, E), generator=g, device="cuda")
    top, ids = torch.topk(logits, k, dim=1)
    ids = ids.to(torch.int32)
    weights = torch.softmax(top, 1)
    slots = torch.where(torch.rand((T, k), generator=g, device="cuda") < c["off"], torch.full_like(ids, -1), ids)
    rows = None
    if c["mapped"]:                                       # rows in (expert, token) order
        order = torch.argsort(ids.reshape(-1).to(torch.int64) * (T * k) + torch.arange(T * k, device="cuda"))
        rows = torch.empty(T * k, dtype=torch.int32, device="cuda")
        rows[order] = torch.arange(T * k, dtype=torch.int32, device="cuda")
    return dict(dout=_randn(g, (T, h), 0.05, torch.bfloat16), y=_randn(g, (T * k, h), 1.0, DT[c["dt"]]), ids=ids,
                slots=slots, weights=weights.contiguous(), route_rows=rows)


def prepare(case, seed):
    c = case
    s = _inputs(case, seed)
    s.pop("counts", None)
    s["case"] = c
    new = lambda shape, dt: torch.empty(shape, dtype=dt, device="cuda")  # noqa: E731
    if c["op"] == "product":
        s["out"] = new((c["rows"], c["n"]), DT[c["out"]])
    elif c["op"] == "wgrad":
        s["dw"] = new((c["experts"], c["n"], c["k"]), DT[c["out"]])
    elif c["op"] == "saved":
        R, n, dt, groups = c["rows"], c["n"], DT[c["dt"]], -(-c["n"] // 128)
        if c["form"] == "use":
            s["dx"] = new((R, 2 * n), dt)
        else:
            both = 2 if c["form"] == "save" else 1
            s["q"] = new((R, both * n), torch.uint8)
            s["s"] = new((R, both * groups), torch.float32)
        if c["form"] != "save_rows":
            s["h"] = new((R, n), dt)
    else:
        s["dy"] = torch.zeros_like(s["y"])                # rows that no active route names stay zero
        s["dweights"] = torch.empty_like(s["weights"])
        s["dlogits"] = new((c["tokens"], c["experts"]), torch.float32)
    return s


# ----------------------------------------------------------- the plain forms

def _pow2_scale(amax):
    """The smallest power of two s with amax / s <= 448 (0 where amax is 0)."""
    m, e = torch.frexp(amax)                              # amax = m 2^e, m in [0.5, 1); 448 = 0.875 * 2^9
    s = torch.ldexp(torch.ones_like(amax), torch.where(m <= 0.875, e - 9, e - 8).clamp(min=-126))
    return torch.where(amax == 0, torch.zeros_like(s), s)


def _save_plain(v):
    rows, n = v.shape
    groups = -(-n // 128)
    p = torch.zeros((rows, groups * 128), dtype=torch.float32, device=v.device)
    p[:, :n] = v
    p = p.view(rows, groups, 128)
    s = _pow2_scale(p.abs().amax(dim=2))
    q = torch.where(s[:, :, None] == 0, torch.zeros_like(p), p / s[:, :, None]).to(torch.float8_e4m3fn)
    return q.view(rows, groups * 128)[:, :n].contiguous(), s


def _read_plain(q, s):
    v = q.view(torch.float8_e4m3fn).float()
    return v * s.repeat_interleave(128, dim=1)[:, :v.shape[1]]


def _gate_plain(act, g):
    """act(g) and its derivative."""
    if act == "silu":
        r = 1 / (1 + torch.exp(-g))
        return g * r, r * (1 + g * (1 - r))
    if act == "gelu":
        p = 0.5 * (1 + torch.erf(g * math.sqrt(0.5)))
        return g * p, p + g * torch.exp(-0.5 * g * g) * (1 / math.sqrt(2 * math.pi))
    if act == "relu":
        on = (g > 0).float()
        return g * on, on
    if act == "sigmoid":
        r = 1 / (1 + torch.exp(-g))
        return r, r * (1 - r)
    return g, torch.ones_like(g)


def _plain(s, c):
    if c["op"] == "product":
        dt = DT[c["out"]]
        if c["form"] == "slot":
            on = s["slots"] >= 0
            token = torch.arange(c["rows"], device="cuda") // c["per_token"]
            w = s["w"][s["slots"].clamp(min=0).long()].float()
            y = (w * s["a"].float()[token][:, None, :]).sum(dim=2)
            return torch.where(on[:, None], y, torch.zeros_like(y)).to(dt)
        a = s["a"].float()[s["pad"]]                      # [E, longest, K]; places past an expert's rows are dropped
        w = s["w"].float()
        y = torch.bmm(a, w.transpose(1, 2) if c["form"] == "forward" else w)
        return y[s["expert"], s["place"]].to(dt)
    if c["op"] == "wgrad":
        a = s["a"].float() if s["a_s"] is None else _read_plain(s["a"], s["a_s"])
        there = s["there"][:, :, None]
        a = torch.where(there, a[s["pad"]], torch.zeros((), device="cuda"))
        dy = torch.where(there, s["dy"].float()[s["pad"]], torch.zeros((), device="cuda"))
        return torch.bmm(dy.transpose(1, 2), a).to(DT[c["out"]])
    if c["op"] == "saved":
        n, dt = c["n"], DT[c["dt"]]
        if c["form"] == "save_rows":
            q, scale = _save_plain(s["x"].float())
            return dict(codes=q, scales=scale)
        if c["form"] == "save":
            x = s["x"].float()
            (qg, sg), (qu, su) = _save_plain(x[:, :n]), _save_plain(x[:, n:])
            h = _gate_plain(c["act"], x[:, :n])[0] * x[:, n:]
            both = torch.cat([qg.view(torch.uint8), qu.view(torch.uint8)], 1).view(torch.float8_e4m3fn)
            return dict(h=h.to(dt), codes=both, scales=torch.cat([sg, su], 1))
        half = s["s"].shape[1] // 2
        gate, up = _read_plain(s["q"][:, :n], s["s"][:, :half]), _read_plain(s["q"][:, n:], s["s"][:, half:])
        f, d = _gate_plain(c["act"], gate)
        dh = s["dh"].float()
        return dict(dx=torch.cat([dh * up * d, dh * f], 1).to(dt), h=(f * up).to(dt))
    T, k = s["slots"].shape
    on = s["slots"] >= 0
    rows = torch.arange(T * k, device="cuda") if s["route_rows"] is None else s["route_rows"].long()
    dout, zero = s["dout"].float(), torch.zeros((), device="cuda")
    dy = torch.zeros(s["y"].shape, dtype=torch.float32, device="cuda")
    dy[rows] = torch.where(on[:, :, None], s["weights"][:, :, None] * dout[:, None, :], zero).view(T * k, -1)
    dw = torch.where(on, (dout[:, None, :] * s["y"][rows].float().view(T, k, -1)).sum(dim=2), zero)
    back = s["weights"] * (dw - (s["weights"] * dw).sum(dim=1, keepdim=True))
    dlogits = torch.zeros((T, c["experts"]), device="cuda").scatter_(1, s["ids"].long(), back)
    return dict(dy=dy.to(s["y"].dtype), dweights=dw, dlogits=dlogits)


# ---------------------------------------------------------------- one pass

def _own(s, c):
    import moe_routed_expert_amd as m
    if c["op"] == "product":
        if c["form"] == "slot":
            m.b16_grouped_gemm(s["a"], s["w"], s["out"], mode=m.MOE_MODE_SLOT, slot_ids=s["slots"],
                               a_row_div=c["per_token"])
        else:
            m.b16_grouped_gemm(s["a"], s["w"], s["out"], mode=m.MOE_MODE_GROUPED, expert_offsets=s["offsets"],
                               w_trans=c["form"] == "data_grad")
        return s["out"]
    if c["op"] == "wgrad":
        m.b16_grouped_wgrad(s["dy"], s["a"], s["offsets"], s["dw"], a_s=s["a_s"])
        return s["dw"]
    if c["op"] == "saved":
        if c["form"] == "use":
            m.gated_act_backward(s["dh"], s["q"], s["s"], s["dx"], act=ACTS[c["act"]], h=s["h"])
            return dict(dx=s["dx"], h=s["h"])
        if c["form"] == "save_rows":
            m.act_checkpoint(s["x"], s["q"], s["s"])
            return dict(codes=s["q"].view(torch.float8_e4m3fn), scales=s["s"])
        m.act_checkpoint(s["x"], s["q"], s["s"], act=ACTS[c["act"]], h=s["h"])
        return dict(h=s["h"], codes=s["q"].view(torch.float8_e4m3fn), scales=s["s"])
    if c["mapped"] and c["off"]:
        s["dy"].zero_()                                   # a step that drops routes clears their rows every time
    m.topk_reduce_backward(s["dout"], s["y"], s["slots"], s["weights"], s["dy"], s["dweights"],
                           route_rows=s["route_rows"])
    m.route_prep_backward(s["ids"], s["weights"], s["dweights"], s["dlogits"])
    return dict(dy=s["dy"], dweights=s["dweights"], dlogits=s["dlogits"])


def run(state):
    return _own(state, state["case"]) if own else _plain(state, state["case"])


# ---------------------------------------------- the definitions in 64 bits

def _exact_codes(v):
    """(codes, scales) of float64 rows: the scale's exponent from amax / 448, codes rounded half to even."""
    rows, n = v.shape
    groups = (n + 127) // 128
    scales = torch.zeros((rows, groups), dtype=torch.float64, device=v.device)
    codes = torch.zeros_like(v)
    for j in range(groups):
        x = v[:, 128 * j:128 * (j + 1)]
        top = x.abs().max(dim=1).values
        m, e = torch.frexp(top / 448)
        s = torch.exp2((e - (m == 0.5).int()).double()).clamp(min=2.0 ** -126)
        t = x / s[:, None]
        step = torch.exp2(torch.frexp(t)[1].clamp(min=-5).double() - 4)   # e4m3: 3 mantissa bits, least exponent -6
        codes[:, 128 * j:128 * (j + 1)] = torch.round(t / step) * step
        scales[:, j] = torch.where(top == 0, torch.zeros_like(s), s)
    return codes, scales


def _exact_act(act, g):
    r = torch.special.expit(g)
    p = torch.special.ndtr(g)
    return {"silu": (g * r, r + g * r * torch.special.expit(-g)),
            "gelu": (g * p, p + g * torch.exp(-g * g / 2) / math.sqrt(2 * math.pi)),
            "relu": (g.clamp(min=0), (g > 0).double()),
            "sigmoid": (r, r * torch.special.expit(-g)),
            "mul": (g, torch.ones_like(g))}[act]


def _exact_values(q, s):
    n = q.shape[1]
    group = torch.arange(n, device=q.device) // 128
    return q.view(torch.float8_e4m3fn).double() * s.double()[:, group]


def exact(case, seed):
    c, d = case, _inputs(case, seed)
    if c["op"] == "product":
        out = torch.zeros((c["rows"], c["n"]), dtype=torch.float64, device="cuda")
        if c["form"] == "slot":
            for r, e in enumerate(d["slots"].tolist()):
                if e >= 0:
                    out[r] = d["w"][e].double() @ d["a"][r // c["per_token"]].double()
            return out
        lo = 0
        for e, cnt in enumerate(d["counts"].tolist()):
            if cnt:
                w = d["w"][e].double()
                out[lo:lo + cnt] = d["a"][lo:lo + cnt].double() @ (w.t() if c["form"] == "forward" else w)
            lo += cnt
        return out
    if c["op"] == "wgrad":
        out = torch.zeros((c["experts"], c["n"], c["k"]), dtype=torch.float64, device="cuda")
        lo = 0
        for e, cnt in enumerate(d["counts"].tolist()):
            if cnt:
                a = d["a"][lo:lo + cnt]
                a = a.double() if d["a_s"] is None else _exact_values(a, d["a_s"][lo:lo + cnt])
                out[e] = d["dy"][lo:lo + cnt].double().t() @ a
            lo += cnt
        return out
    if c["op"] == "saved":
        n = c["n"]
        if c["form"] == "save_rows":
            q, s = _exact_codes(d["x"].double())
            return dict(codes=q, scales=s)
        if c["form"] == "save":
            x = d["x"].double()
            (qg, sg), (qu, su) = _exact_codes(x[:, :n]), _exact_codes(x[:, n:])
            return dict(h=_exact_act(c["act"], x[:, :n])[0] * x[:, n:], codes=torch.cat([qg, qu], 1),
                        scales=torch.cat([sg, su], 1))
        half = d["s"].shape[1] // 2
        gate, up = _exact_values(d["q"][:, :n], d["s"][:, :half]), _exact_values(d["q"][:, n:], d["s"][:, half:])
        f, df = _exact_act(c["act"], gate)
        dh = d["dh"].double()
        return dict(dx=torch.cat([dh * up * df, dh * f], 1), h=f * up)
    T, k = d["slots"].shape
    dout, w = d["dout"].double(), d["weights"].double()
    dy = torch.zeros(d["y"].shape, dtype=torch.float64, device="cuda")
    dw = torch.zeros((T, k), dtype=torch.float64, device="cuda")
    for j in range(k):
        on = (d["slots"][:, j] >= 0).double()
        rows = torch.arange(T, device="cuda") * k + j
        if d["route_rows"] is not None:
            rows = d["route_rows"].long()[rows]
        dy[rows] = (w[:, j] * on)[:, None] * dout
        dw[:, j] = on * (dout * d["y"][rows].double()).sum(dim=1)
    mean = (w * dw).sum(dim=1)
    dlogits = torch.zeros((T, c["experts"]), dtype=torch.float64, device="cuda")
    for j in range(k):
        dlogits[torch.arange(T, device="cuda"), d["ids"][:, j].long()] = w[:, j] * (dw[:, j] - mean)
    return dict(dy=dy, dweights=dw, dlogits=dlogits)
