"""What is measured of the router with its gradient and of the experts' products in microscaled 4-bit floating point.

Five operators, each in its directions and types:

  route      scores (softmax or sigmoid), a bias that takes part in the choice only, groups, top-k, weights, and the
             maps of the routes in (expert, token) order.  A logit of -inf masks its expert for that token; a token
             whose experts are all masked (a padded batch) takes no route.
  route_grad the logits' gradient from the weights' and, for an auxiliary loss, the scores'.
  quantise   rows (or act(gate) * up of them) to MXFP4, 32 codes a power-of-two scale, and read back as values.
  product    out[r] = a[r] @ W[e(r)]^T with MXFP4 on both sides, rows grouped by expert (ragged); "slot" is the
             decode form: each route names its expert's slot, a negative slot gives a zero row.
  experts    the routed experts in MXFP4 as they are used: tokens quantised, gate/up with activation and requant, down.
"""
import math

import numpy as np
import torch

own = False

DT = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
ACTS = {"none": 0, "silu": 1, "gelu": 2, "relu": 3, "sigmoid": 4, "mul": 5}


# ---------------------------------------------------------------- the cases

def listed():
    return [
        # a prefill of 4096 tokens, sigmoid scores with a balance bias, four of eight groups stay
        dict(name="route_prefill_groups", op="route", dt="fp32", tokens=4096, experts=256, topk=8, score="sigmoid",
             bias=True, groups=8, keep=4, top=2, renorm=True, scale=2.5, scores=False, masked=0.0),
        # a decode step of eight tokens over a pool of 64 experts, 16-bit logits with ties
        dict(name="route_decode", op="route", dt="bf16", tokens=8, experts=64, topk=8, score="softmax", bias=False,
             groups=1, keep=1, top=1, renorm=False, scale=1.0, scores=False, masked=0.0),
        # a large padded training batch, scores kept for the auxiliary loss
        dict(name="route_padded_e512", op="route", dt="bf16", tokens=16384, experts=512, topk=6, score="softmax",
             bias=True, groups=1, keep=1, top=1, renorm=True, scale=1.0, scores=True, masked=0.1),
        # its backward at prefill size: weights that are not renormalised, an auxiliary loss whose gradient is one row
        dict(name="route_grad_aux", op="route_grad", dt="fp32", tokens=4096, experts=256, topk=6, score="softmax",
             renorm=False, scale=1.0, aux="row", masked=0.0),
        # an odd batch over an odd number of experts
        dict(name="route_grad_odd", op="route_grad", dt="bf16", tokens=333, experts=100, topk=5, score="sigmoid",
             renorm=True, scale=1.5, aux="none", masked=0.05),
        # the gathered rows of a 24576-route step
        dict(name="quantise_rows", op="quantise", act="none", rule="floor", dt="bf16", rows=24576, n=4096),
        # a few routes of a small expert, the width ends inside a group
        dict(name="quantise_act_small", op="quantise", act="silu", rule="ceil", dt="fp16", rows=37, n=712),
        # few large experts: the matrix units bound it
        dict(name="product_e8", op="product", form="grouped", out="bf16", experts=8, rows=16384, skew=0.1, n=4096,
             k=8192),
        # a short ragged batch with widths that fit no tile, some experts empty
        dict(name="product_ragged_odd", op="product", form="grouped", out="fp16", experts=16, rows=333, skew=1.5,
             n=1000, k=544),
        # one token's eight routes against a pool of 64 resident experts, one inactive
        dict(name="product_slot_decode", op="product", form="slot", out="fp32", experts=64, rows=8, per_token=8, off=1,
             n=1536, k=2048),
        # a prefill of 4096 tokens over 256 experts, six each: the experts' weights dominate
        dict(name="experts_prefill_e256", op="experts", form="grouped", act="silu", experts=256, tokens=4096, topk=6,
             off=0, h=4096, i=1024),
        # one token's decode step
        dict(name="experts_decode", op="experts", form="slot", act="silu", experts=64, tokens=1, topk=8, off=0, h=2048,
             i=768),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _log_of(rng, step, lo, hi):
    return step * max(1, _log(rng, lo / step, hi / step))


def draw(rng):
    while True:
        op = rng.choice(["route", "route", "route_grad", "quantise", "product", "product", "product", "experts", "experts"])
        if op in ("route", "route_grad"):
            experts = _log(rng, 8, 1024)
            c = dict(op=op, dt=rng.choice(["bf16", "fp16", "fp32"]), tokens=_log(rng, 1, 32768), experts=experts,
                     topk=rng.randint(1, 8), score=rng.choice(["softmax", "sigmoid"]), renorm=rng.random() < 0.5,
                     scale=rng.choice([1.0, 2.5]), masked=rng.choice([0.0, 0.1]))
            if op == "route_grad":
                c["aux"] = rng.choice(["none", "row", "full"])
            else:
                c.update(bias=rng.random() < 0.6, groups=1, keep=1, top=1, scores=rng.random() < 0.3)
                if rng.random() < 0.4:
                    groups = rng.choice([2, 4, 8])
                    c.update(experts=groups * max(2, experts // groups), groups=groups, keep=rng.randint(1, groups),
                             top=rng.choice([1, 2]))
                c["topk"] = min(c["topk"], c["keep"] * (c["experts"] // c["groups"]))
        elif op == "quantise":
            c = dict(op=op, act=rng.choice(["none", "none", "relu", "mul"]), rule=rng.choice(["floor", "ceil"]),
                     dt=rng.choice(["bf16", "fp16", "fp32"]), rows=_log(rng, 1, 24576), n=_log_of(rng, 2, 32, 8192))
            if c["rows"] * c["n"] < 3e5:                  # transcendental gates: few values next to a code's border
                c["act"] = rng.choice(sorted(ACTS))
        elif op == "product":
            c = dict(op=op, form=rng.choice(["grouped", "grouped", "slot"]), out=rng.choice(["bf16", "fp16", "fp32"]),
                     n=_log_of(rng, 8, 64, 8192), k=_log_of(rng, 32, 64, 8192))
            if c["form"] == "slot":
                per = rng.choice([1, 2, 6, 8])
                c.update(experts=_log(rng, 1, 64), rows=per * _log(rng, 1, 8), per_token=per, off=rng.choice([0, 1]))
            else:
                c.update(experts=_log(rng, 1, 256), rows=_log(rng, 1, 24576), skew=rng.uniform(0.0, 1.0))
        else:
            form = rng.choice(["grouped", "slot"])
            experts = _log(rng, 8, 256)
            c = dict(op=op, form=form, act=rng.choice(["silu", "gelu", "relu", "sigmoid", "mul"]), experts=experts,
                     tokens=_log(rng, 1, 8) if form == "slot" else _log(rng, 1, 4096), topk=rng.choice([1, 2, 6, 8]),
                     off=rng.choice([0, 1]) if form == "slot" else 0, h=_log_of(rng, 32, 128, 8192),
                     i=_log_of(rng, 32, 64, 2048))
        w = work(c)
        most = {"route": 6e7, "route_grad": 6e7, "quantise": 5.5e8}.get(op, 1.8e9)
        if w["flops"] <= 1.1e12 and w["bytes"] <= most:
            return c


def _mx(elements):
    """Bytes of so many MXFP4 elements: a code of half a byte, a scale byte for 32."""
    return elements // 2 + elements // 32


def _used(E, R):
    """Experts that some of R rows name."""
    return E * (1.0 - (1.0 - 1.0 / E) ** R)


def work(case):
    c = case
    if c["op"] in ("route", "route_grad"):
        T, E, k = c["tokens"], c["experts"], c["topk"]
        size = 4 if c["dt"] == "fp32" else 2
        if c["op"] == "route_grad":
            aux = {"none": 0, "row": 4 * E, "full": 4 * T * E}[c["aux"]]
            return dict(bytes=2 * T * E * size + 12 * T * k + aux, flops=10 * T * E)
        return dict(bytes=T * E * (size + (4 if c["scores"] else 0)) + 16 * T * k + 4 * (E + 1), flops=10 * T * E)
    if c["op"] == "quantise":
        R, n, size = c["rows"], c["n"], 4 if c["dt"] == "fp32" else 2
        codes = R * (n // 2 + -(-n // 32))
        return dict(bytes=R * n * size * (1 if c["act"] == "none" else 2) + 2 * codes + 2 * R * n, flops=8 * R * n)
    if c["op"] == "product":
        R, E, n, k = c["rows"], c["experts"], c["n"], c["k"]
        a = R
        if c["form"] == "slot":
            a, R = -(-c["rows"] // c["per_token"]), R - c["off"]
        size = 4 if c["out"] == "fp32" else 2
        return dict(bytes=int(_mx(a * k) + _used(E, R) * _mx(n * k) + c["rows"] * n * size), flops=2 * R * n * k)
    T, E, h, i = c["tokens"], c["experts"], c["h"], c["i"]
    R = T * min(c["topk"], E)
    used = _used(E, R - c["off"])
    return dict(bytes=int(T * h * 2 + used * _mx(3 * h * i) + R * h * 2), flops=6 * R * h * i)


# --------------------------------------------------------------- the inputs

def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed & 0x7FFFFFFFFFFF)
    return g


def _randn(g, shape, std, dt):
    return (torch.randn(shape, generator=g, device="cuda", dtype=torch.float32) * std).to(dt)


def _mx_bank(g, shape, std):
    """Normal values in MXFP4: packed codes and scale bytes, drawn in pieces so that a bank needs no 32-bit copy."""
    *lead, k = shape
    rows = math.prod(lead)
    q = torch.empty((rows, k // 2), dtype=torch.uint8, device="cuda")
    s = torch.empty((rows, k // 32), dtype=torch.uint8, device="cuda")
    step = max(1, (1 << 27) // k)
    for r in range(0, rows, step):
        x = torch.randn((min(step, rows - r), k), generator=g, device="cuda") * std
        e = torch.frexp(x.abs().view(-1, k // 32, 32).amax(dim=2))[1] - 3
        t = torch.ldexp(x.view(-1, k // 32, 32), -e[:, :, None]).view(-1, k)
        sign, t = (t < 0).to(torch.uint8) * 8, t.abs()
        for border in (0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0):
            sign += t > border
        q[r:r + step] = sign[:, 0::2] + 16 * sign[:, 1::2]
        s[r:r + step] = (e + 127).to(torch.uint8)
    return q.view(*lead, k // 2), s.view(*lead, k // 32)


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
    dev = lambda x: torch.from_numpy(np.ascontiguousarray(x)).cuda()  # noqa: E731
    return dict(offsets=dev(offs), expert=dev(expert.astype(np.int64)), place=dev(place.astype(np.int64)),
                pad=dev(pad.astype(np.int64)))


def _logits(c, g):
    T, E, dt = c["tokens"], c["experts"], DT[c["dt"]]
    x = torch.randn((T, E), generator=g, device="cuda") * 1.5 + torch.randn(E, generator=g, device="cuda") * 0.5
    if c["masked"]:
        x = x.masked_fill(torch.rand(E, generator=g, device="cuda") < c["masked"] / 4, -math.inf)   # experts that are away
        x = x.masked_fill(torch.rand((T, 1), generator=g, device="cuda") < c["masked"], -math.inf)  # padding
    return x.to(dt)


def _slots(c, rows, seed):
    rng = np.random.default_rng(seed)
    slots = rng.integers(0, c["experts"], size=rows).astype(np.int32)
    if c["off"] and rows > 1:
        slots[rng.integers(0, rows)] = -1
    return torch.from_numpy(slots).cuda()


def _inputs(case, seed):
    c, g = case, _gen(seed)
    if c["op"] == "route":
        bias = _randn(g, (c["experts"],), 0.05, torch.float32) if c["bias"] else None
        return dict(logits=_logits(c, g), bias=bias)
    if c["op"] == "route_grad":
        logits = _logits(c, g)
        T, k = c["tokens"], min(c["topk"], c["experts"])
        top, ids = torch.topk(torch.nan_to_num(logits.float(), neginf=-1e30), k, dim=1)
        ids = torch.where(top > -1e29, ids, -1).to(torch.int32)
        x = logits.double()
        s = torch.sigmoid(x) if c["score"] == "sigmoid" else torch.softmax(x, 1).nan_to_num(0.0)
        w = torch.where(ids >= 0, s.gather(1, ids.clamp(min=0).long()), 0.0)
        if c["renorm"]:
            w = w / w.sum(dim=1, keepdim=True).clamp(min=1e-300)
        dscores = None
        if c["aux"] != "none":
            dscores = _randn(g, (1 if c["aux"] == "row" else T, c["experts"]), 0.01, torch.float32).expand(T, -1)
        return dict(logits=logits, ids=ids, weights=(w * c["scale"]).float(),
                    dweights=_randn(g, (T, k), 0.1, torch.float32), dscores=dscores)
    if c["op"] == "quantise":
        return dict(x=_randn(g, (c["rows"], c["n"] * (1 if c["act"] == "none" else 2)), 1.3, DT[c["dt"]]))
    if c["op"] == "product":
        R, slot = c["rows"], c["form"] == "slot"
        rows = -(-R // c["per_token"]) if slot else R
        a, a_s = _mx_bank(g, (rows, c["k"]), 1.0)
        w, w_s = _mx_bank(g, (c["experts"], c["n"], c["k"]), 0.02)
        d = dict(a=a, a_s=a_s, w=w, w_s=w_s)
        if slot:
            return dict(d, slots=_slots(c, R, seed))
        counts = _counts(c, seed)
        return dict(d, counts=counts, **_groups(counts))
    T, E, k, h, i = c["tokens"], c["experts"], min(c["topk"], c["experts"]), c["h"], c["i"]
    d = dict(x=_randn(g, (T, h), 1.0, torch.bfloat16))
    d["w13"], d["w13_s"] = _mx_bank(g, (E, 2 * i, h), 0.02)
    d["w2"], d["w2_s"] = _mx_bank(g, (E, h, i), 0.02)
    if c["form"] == "slot":
        return dict(d, slots=_slots(c, T * k, seed))
    ids = torch.topk(torch.rand((T, E), generator=g, device="cuda"), k, dim=1)[1].reshape(-1)
    order = torch.argsort(ids * (T * k) + torch.arange(T * k, device="cuda"))
    counts = torch.bincount(ids, minlength=E).cpu().numpy()
    return dict(d, source=(order // k).to(torch.int32), counts=counts, **_groups(counts))


def prepare(case, seed):
    c = case
    s = _inputs(case, seed)
    s.pop("counts", None)
    s["case"] = c
    new = lambda shape, dt: torch.empty(shape, dtype=dt, device="cuda")  # noqa: E731
    if c["op"] == "route":
        T, k, i32 = c["tokens"], c["topk"], torch.int32
        s["route"] = (new((T, k), i32), new((T, k), torch.float32), new(T * k, i32), new(T * k, i32),
                      new(c["experts"] + 1, i32), new((T, c["experts"]), torch.float32) if c["scores"] else None)
    elif c["op"] == "route_grad":
        s["dlogits"] = torch.empty_like(s["logits"])
    elif c["op"] == "quantise":
        s["q"], s["s"] = new((c["rows"], c["n"] // 2), torch.uint8), new((c["rows"], -(-c["n"] // 32)), torch.uint8)
        s["values"] = new((c["rows"], c["n"]), torch.bfloat16)
    elif c["op"] == "product":
        s["out"] = new((c["rows"], c["n"]), DT[c["out"]])
    elif c["op"] == "experts":
        T, R, h, i = c["tokens"], c["tokens"] * min(c["topk"], c["experts"]), c["h"], c["i"]
        s["xq"], s["xs"] = new((T, h // 2), torch.uint8), new((T, -(-h // 128) * 4), torch.uint8)[:, :h // 32]
        s["hq"], s["hs"] = new((R, i // 2), torch.uint8), new((R, -(-i // 128) * 4), torch.uint8)[:, :i // 32]
        s["out"] = new((R, h), torch.bfloat16)
    if c["op"] in ("product", "experts"):                 # scale rows begin at multiples of four bytes
        for name in ("a_s", "w_s", "w13_s", "w2_s"):
            if name in s:
                n = s[name].shape[-1]
                s[name] = torch.nn.functional.pad(s[name], (0, -n % 4))[..., :n]
    return s


# ----------------------------------------------------------- the plain forms

E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0, -0.0, -0.5, -1.0, -1.5, -2.0, -3.0, -4.0, -6.0)


def _read_plain(q, s):
    """Packed codes [..., k / 2] and scale bytes [..., k / 32] as fp32 values."""
    t = torch.tensor(E2M1, device="cuda")
    pairs = torch.stack([t.repeat(16), t.repeat_interleave(16)], dim=1)
    v = pairs[q.int()].view(*q.shape[:-1], -1)
    scale = torch.ldexp(torch.ones((), device="cuda"), s.int() - 127)
    v.view(*s.shape, 32).mul_(scale[..., None])
    return v


def _quantise_plain(v, rule):
    """fp32 rows as the values that their MXFP4 form stands for, and the scales."""
    rows, n = v.shape
    groups = -(-n // 32)
    p = torch.nn.functional.pad(v, (0, groups * 32 - n)).view(rows, groups, 32)
    m, e = torch.frexp(p.abs().amax(dim=2))                # amax = m 2^e, m in [0.5, 1)
    e = e - 3 if rule == "floor" else torch.where(m <= 0.75, e - 3, e - 2)   # 6 = 0.75 * 2^3
    e = torch.where(m == 0, -127, e.clamp(min=-127))[:, :, None]
    t = torch.ldexp(p, -e)
    step = torch.ldexp(torch.ones((), device="cuda"), torch.frexp(t)[1].clamp(min=1) - 2)
    t = (torch.round(t / step) * step).clamp(-6.0, 6.0)
    return torch.ldexp(t, e).view(rows, groups * 32)[:, :n], torch.ldexp(torch.ones((), device="cuda"), e[:, :, 0])


def _gate_plain(act, x):
    if act == "none":
        return x
    g, u = x.chunk(2, dim=1)
    f = {"silu": lambda: g / (1 + torch.exp(-g)), "gelu": lambda: g * (0.5 * (1 + torch.erf(g * math.sqrt(0.5)))),
         "relu": lambda: torch.where(g > 0, g, torch.zeros_like(g)), "sigmoid": lambda: 1 / (1 + torch.exp(-g)),
         "mul": lambda: g}[act]()
    return f * u


def _scores_plain(c, logits):
    """Scores in 64 bits, and where an expert may be chosen."""
    x = logits.double()
    there = x > -math.inf
    x = torch.where(there, x, -math.inf)
    if c["score"] == "sigmoid":
        return 1 / (1 + torch.exp(-x)), there
    e = torch.exp(x - x.amax(dim=1, keepdim=True).clamp(min=-1e300))
    return e / e.sum(dim=1, keepdim=True).clamp(min=1e-300), there


def _route_plain(s, c):
    T, E, k = c["tokens"], c["experts"], c["topk"]
    scores, there = _scores_plain(c, s["logits"])
    zero = torch.zeros((), dtype=torch.float64, device="cuda")
    by = scores + s["bias"] if c["bias"] else (s["logits"].double() if c["groups"] == 1 or c["top"] == 1 else scores)
    by = torch.where(there, by, -math.inf)
    if c["groups"] > 1:
        best = by.view(T, c["groups"], -1).sort(dim=2, descending=True)[0][:, :, :c["top"]]
        value = torch.where(best[:, :, 0] > -math.inf, torch.where(best > -math.inf, best, zero).sum(dim=2), -math.inf)
        kept = value.sort(dim=1, descending=True, stable=True)[1][:, :c["keep"]]
        stays = torch.zeros((T, c["groups"]), dtype=torch.bool, device="cuda").scatter_(1, kept, True)
        there = there & stays.repeat_interleave(E // c["groups"], dim=1)
        if not c["bias"]:
            by = s["logits"].double()                     # within the groups the scores' order is the logits'
        by = torch.where(there, by, -math.inf)
    top, ids = by.sort(dim=1, descending=True, stable=True)
    on = top[:, :k] > -math.inf
    ids = torch.where(on, ids[:, :k], -1)
    w = torch.where(on, scores.gather(1, ids.clamp(min=0)), zero)
    if c["renorm"]:
        w = w / w.sum(dim=1, keepdim=True).clamp(min=1e-300)
    flat = ids.reshape(-1)
    key = torch.where(flat >= 0, flat, E)
    order = torch.sort(key, stable=True)[1]               # routes in (expert, token) order, inactive ones last
    count = torch.bincount(key, minlength=E + 1)
    offsets = torch.cat([torch.zeros(1, dtype=torch.int64, device="cuda"), count[:E].cumsum(0)])
    place = torch.empty_like(order).scatter_(0, order, torch.arange(T * k, device="cuda"))
    source = torch.where(torch.arange(T * k, device="cuda") < offsets[E], order // k, -1)
    rows = torch.where(flat >= 0, place, -1)
    out = dict(ids=ids.int(), weights=(w * c["scale"]).float(), dst2src=source.int(), route_rows=rows.int(),
               offsets=offsets.int())
    if c["scores"]:
        out["scores"] = scores.float()
    return out


def _route_grad_plain(s, c):
    scores, there = _scores_plain(c, s["logits"])
    on = s["ids"] >= 0
    ids = s["ids"].clamp(min=0).long()
    g = torch.where(on, s["dweights"].double(), 0.0)
    if c["renorm"]:
        wn = torch.where(on, s["weights"].double() / c["scale"], 0.0)
        back = c["scale"] * wn * (g - (wn * g).sum(dim=1, keepdim=True))
        if c["score"] == "sigmoid":
            back = back * (1 - scores.gather(1, ids))
        dl = torch.zeros_like(scores).scatter_add_(1, ids, back)
        ds = torch.zeros_like(scores)
    else:
        dl = torch.zeros_like(scores)
        ds = torch.zeros_like(scores).scatter_add_(1, ids, c["scale"] * g)
    if s["dscores"] is not None:
        ds = ds + s["dscores"]
    if c["score"] == "sigmoid":
        dl = dl + ds * scores * (1 - scores)
    else:
        dl = dl + scores * (ds - (scores * ds).sum(dim=1, keepdim=True))
    return torch.where(there, dl, 0.0).to(DT[c["dt"]])


def _grouped_plain(a, w, s):
    """a [rows, K] times each row's expert of w [E, N, K], through a padded [E, longest, K] form."""
    return torch.bmm(a[s["pad"]], w.transpose(1, 2))[s["expert"], s["place"]]


def _slot_plain(a, w_of, slots):
    """a [rows, K] against its slot of the bank that w_of(slots) reads; a negative slot gives zeros."""
    y = (w_of(slots.clamp(min=0).long()) * a[:, None, :]).sum(dim=2)
    return torch.where((slots >= 0)[:, None], y, torch.zeros_like(y))


def _plain(s, c):
    if c["op"] == "route":
        return _route_plain(s, c)
    if c["op"] == "route_grad":
        return _route_grad_plain(s, c)
    if c["op"] == "quantise":
        v, scale = _quantise_plain(_gate_plain(c["act"], s["x"].float()), c["rule"])
        return dict(values=v.to(torch.bfloat16), scales=scale.to(torch.float8_e8m0fnu))
    if c["op"] == "product":
        a = _read_plain(s["a"], s["a_s"])
        if c["form"] == "slot":
            a = a[torch.arange(c["rows"], device="cuda") // c["per_token"]]
            return _slot_plain(a, lambda e: _read_plain(s["w"][e], s["w_s"][e]), s["slots"]).to(DT[c["out"]])
        return _grouped_plain(a, _read_plain(s["w"], s["w_s"]), s).to(DT[c["out"]])
    x = _quantise_plain(s["x"].float(), "floor")[0]
    if c["form"] == "slot":
        x = x.repeat_interleave(min(c["topk"], c["experts"]), dim=0)
        y = _slot_plain(x, lambda e: _read_plain(s["w13"][e], s["w13_s"][e]), s["slots"])
        h = _quantise_plain(_gate_plain(c["act"], y), "floor")[0]
        return _slot_plain(h, lambda e: _read_plain(s["w2"][e], s["w2_s"][e]), s["slots"]).to(torch.bfloat16)
    y = _grouped_plain(x[s["source"].long()], _read_plain(s["w13"], s["w13_s"]), s)
    h = _quantise_plain(_gate_plain(c["act"], y), "floor")[0]
    return _grouped_plain(h, _read_plain(s["w2"], s["w2_s"]), s).to(torch.bfloat16)


# ---------------------------------------------------------------- one pass

def _own(s, c):
    import moe_routed_expert_amd as m
    score = {"softmax": 0, "sigmoid": 1}.get(c.get("score"))
    if c["op"] == "route":
        r = m.router(s["logits"], c["topk"], score=score, bias=s["bias"], n_group=c["groups"], topk_group=c["keep"],
                     group_top=c["top"], renorm=c["renorm"], scale=c["scale"], out=s["route"])
        out = dict(ids=r.expert_ids, weights=r.weights, dst2src=r.dst2src, route_rows=r.route_rows,
                   offsets=r.expert_offsets)
        if c["scores"]:
            out["scores"] = r.scores
        return out
    if c["op"] == "route_grad":
        m.router_backward(s["logits"], s["ids"], s["weights"], s["dweights"], s["dlogits"], score=score,
                          renorm=c["renorm"], scale=c["scale"], dscores=s["dscores"])
        return s["dlogits"]
    if c["op"] == "quantise":
        m.mx4_quant(s["x"], s["q"], s["s"], act=ACTS[c["act"]], rule={"floor": 0, "ceil": 1}[c["rule"]])
        m.mx4_dequant(s["q"], s["s"], s["values"])
        return dict(values=s["values"], scales=s["s"].view(torch.float8_e8m0fnu))
    slot = c["form"] == "slot"
    if c["op"] == "product":
        how = (dict(mode=m.MOE_MODE_SLOT, slot_ids=s["slots"], a_row_div=c["per_token"]) if slot
               else dict(mode=m.MOE_MODE_GROUPED, expert_offsets=s["offsets"]))
        m.mx4_grouped_gemm(s["a"], s["a_s"], s["w"], s["w_s"], s["out"], **how)
        return s["out"]
    m.mx4_quant(s["x"], s["xq"], s["xs"])
    if slot:
        how = dict(mode=m.MOE_MODE_SLOT, slot_ids=s["slots"])
        first = dict(how, a_row_div=min(c["topk"], c["experts"]))
    else:
        how = dict(mode=m.MOE_MODE_GROUPED, expert_offsets=s["offsets"])
        first = dict(how, a_rows=s["source"])
    m.mx4_grouped_gemm_act_quant(s["xq"], s["xs"], s["w13"], s["w13_s"], s["hq"], s["hs"], act=ACTS[c["act"]], **first)
    m.mx4_grouped_gemm(s["hq"], s["hs"], s["w2"], s["w2_s"], s["out"], **how)
    return s["out"]


def run(state):
    return _own(state, state["case"]) if own else _plain(state, state["case"])


# ---------------------------------------------- the definitions in 64 bits

def _exact_values(q, s):
    """Codes as sign, exponent and mantissa bits: (-1)^s 2^(e-1) (1 + m/2), or m/2 where e is 0; times the scale."""
    code = torch.stack([q & 15, q >> 4], dim=-1).reshape(*q.shape[:-1], -1).long()
    e, m = (code >> 1) & 3, (code & 1).double()
    mag = torch.where(e == 0, m / 2, torch.exp2((e - 1).double()) * (1 + m / 2))
    group = torch.arange(code.shape[-1], device=q.device) // 32
    return torch.where(code >= 8, -mag, mag) * torch.exp2(s.double() - 127)[..., group]


def _exact_quantise(v, rule):
    """(values, scales) of float64 rows: the nearest of the format's values, ties to the even mantissa."""
    grid = torch.tensor([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0], dtype=torch.float64, device=v.device)
    even = torch.tensor([0, 2, 2, 4, 4, 6, 6], device=v.device)      # of two neighbours, the one with mantissa bit 0
    values, scales = torch.zeros_like(v), []
    for j in range(0, v.shape[1], 32):
        x = v[:, j:j + 32]
        top = x.abs().max(dim=1).values
        safe = top.clamp(min=2.0 ** -200)
        e = torch.floor(torch.log2(safe)) - 2 if rule == "floor" else torch.ceil(torch.log2(safe / 6))
        two = lambda n: torch.exp2(n)  # noqa: E731
        if rule == "floor":                                # the logarithm may round across a power of two
            e = torch.where(two(e + 2) > safe, e - 1, torch.where(two(e + 3) <= safe, e + 1, e))
        else:
            e = torch.where(6 * two(e) < safe, e + 1, torch.where(6 * two(e - 1) >= safe, e - 1, e))
        s = two(torch.where(top == 0, -127.0, e.clamp(min=-127)))
        t = (x.abs() / s[:, None]).clamp(max=6.0)
        low = (torch.searchsorted(grid, t.contiguous(), right=True) - 1).clamp(max=6)
        a, b = grid[low], grid[low + 1]
        code = torch.where(t - a < b - t, low, torch.where(t - a > b - t, low + 1, even[low]))
        values[:, j:j + 32] = torch.sign(x) * grid[code] * s[:, None]
        scales.append(s)
    return values, torch.stack(scales, dim=1)


def _exact_gate(act, x):
    if act == "none":
        return x
    n = x.shape[1] // 2
    g, u = x[:, :n], x[:, n:]
    f = {"silu": lambda: g * torch.special.expit(g), "gelu": lambda: g * torch.special.ndtr(g),
         "relu": lambda: g.clamp(min=0), "sigmoid": lambda: torch.special.expit(g), "mul": lambda: g}
    return f[act]() * u


def _exact_scores(c, x):
    if c["score"] == "sigmoid":
        return torch.special.expit(x)
    return torch.exp(torch.log_softmax(x, dim=1)).nan_to_num(0.0)


def _exact_route(c, d):
    T, E, k, G = c["tokens"], c["experts"], c["topk"], c["groups"]
    x = d["logits"].double()
    s = _exact_scores(c, x)
    gone = torch.isinf(x)
    choice = (s + d["bias"].double()) if c["bias"] else s
    rank = choice if c["bias"] else x
    if G > 1:
        left, value = torch.where(gone, -math.inf, choice if c["top"] == 2 else rank).view(T, G, E // G).clone(), None
        for _ in range(c["top"]):
            top = left.max(dim=2, keepdim=True)
            value = top.values[:, :, 0] if value is None else value + top.values[:, :, 0].clamp(min=-1e308).where(
                top.values[:, :, 0] > -math.inf, torch.zeros((), dtype=torch.float64, device="cuda"))
            left.scatter_(2, top.indices, -math.inf)
        out = torch.ones((T, G), dtype=torch.bool, device="cuda")
        for _ in range(c["keep"]):
            best = value.argmax(dim=1, keepdim=True)
            out.scatter_(1, best, False)
            value = value.scatter(1, best, -math.inf)
        gone = gone | out[:, torch.arange(E, device="cuda") // (E // G)]
    left = torch.where(gone, -math.inf, rank)
    chosen = []
    for _ in range(k):
        top = left.max(dim=1, keepdim=True)
        w = s.gather(1, top.indices)
        chosen.append(torch.where(top.values > -math.inf, w, 0.0))
        left.scatter_(1, top.indices, -math.inf)
    w = torch.cat(chosen, dim=1)
    if c["renorm"]:
        total = w.sum(dim=1, keepdim=True)
        w = torch.where(total > 0, w / total, 0.0)
    out = dict(ids=None, weights=w * c["scale"], dst2src=None, route_rows=None, offsets=None)
    if c["scores"]:
        out["scores"] = s
    return out


def _exact_route_grad(c, d):
    """Reverse-mode differentiation of the weights (and the auxiliary loss) in 64 bits."""
    x = d["logits"].double()
    gone = torch.isinf(x)
    leaf = torch.where(gone, 0.0, x).requires_grad_()
    with torch.enable_grad():
        shown = leaf.masked_fill(gone, -1e30)
        s = torch.sigmoid(shown) if c["score"] == "sigmoid" else torch.softmax(shown, dim=1)
        on = d["ids"] >= 0
        w = s.gather(1, d["ids"].clamp(min=0).long()).masked_fill(~on, 0.0)
        if c["renorm"]:
            total = w.sum(dim=1, keepdim=True)
            w = w / torch.where(total > 0, total, 1.0)
        loss = (c["scale"] * w * d["dweights"].double()).sum()
        if d["dscores"] is not None:
            loss = loss + (s.masked_fill(gone, 0.0) * d["dscores"].double()).sum()
        return torch.autograd.grad(loss, leaf)[0].masked_fill(gone, 0.0)


def exact(case, seed):
    c, d = case, _inputs(case, seed)
    if c["op"] == "route":
        return _exact_route(c, d)
    if c["op"] == "route_grad":
        return _exact_route_grad(c, d)
    if c["op"] == "quantise":
        v, scale = _exact_quantise(_exact_gate(c["act"], d["x"].double()), c["rule"])
        return dict(values=v, scales=scale)
    if c["op"] == "product":
        out = torch.zeros((c["rows"], c["n"]), dtype=torch.float64, device="cuda")
        a = _exact_values(d["a"], d["a_s"])
        if c["form"] == "slot":
            for r, e in enumerate(d["slots"].tolist()):
                if e >= 0:
                    out[r] = _exact_values(d["w"][e], d["w_s"][e]) @ a[r // c["per_token"]]
            return out
        at = 0
        for e, n in enumerate(d["counts"].tolist()):
            if n:
                out[at:at + n] = a[at:at + n] @ _exact_values(d["w"][e], d["w_s"][e]).t()
            at += n
        return out
    x = _exact_quantise(d["x"].double(), "floor")[0]
    k = min(c["topk"], c["experts"])
    out = torch.zeros((c["tokens"] * k, c["h"]), dtype=torch.float64, device="cuda")

    def expert(e, rows):
        y = rows @ _exact_values(d["w13"][e], d["w13_s"][e]).t()
        return _exact_quantise(_exact_gate(c["act"], y), "floor")[0] @ _exact_values(d["w2"][e], d["w2_s"][e]).t()

    if c["form"] == "slot":
        for r, e in enumerate(d["slots"].tolist()):
            if e >= 0:
                out[r] = expert(e, x[r // k][None, :])[0]
        return out
    at, source = 0, d["source"].long()
    for e, n in enumerate(d["counts"].tolist()):
        if n:
            out[at:at + n] = expert(e, x[source[at:at + n]])
        at += n
    return out
