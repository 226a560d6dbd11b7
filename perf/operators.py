"""The optimizer step over a list of tensors: what is computed, on what sizes.

Three operators, each over every parameter tensor of a model at once:

  norm    the global norm of the gradients, the clip coefficient and the
          non-finite flag
  adamw   one AdamW update, with fp32 moments ("state": 32) or with moments
          in 8 bits per element ("state": 8)
  pack    fp32 or bf16 moments to 8 bits (returned as the values the codes
          stand for), and unpack, the way back

A model here is the usual decoder: two vocab x d matrices, and per layer
four d x d and three ffn x d matrices and two vectors of d, plus one vector.
Matrices have the case's param dtype, vectors are fp32 and take no weight
decay; a 16-bit param has an fp32 master copy.  The tensors are views of one
flat buffer per dtype, each starting at a multiple of `pad` elements (pad 1:
at any element), so whole-buffer torch operations compute the plain form and
the tensors' list is what the framework's own calls take.
"""

import math

import numpy as np
import torch

own = False

BLOCK = 256
DT = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
SIZE = {"f32": 4, "bf16": 2, "f16": 2}
B1, B2, EPS, LR, WD = 0.9, 0.95, 1e-8, 1e-4, 0.1
MAX_NORM = 1.0
SEED = 1234567  # of the stochastic rounding
M32 = 0xFFFFFFFF


def listed():
    tiny = dict(layers=2, d=96, ffn=256, vocab=1001)
    odd = dict(layers=12, d=769, ffn=2051, vocab=30011)
    big = dict(layers=24, d=2048, ffn=5504, vocab=32000)
    return [
        # a few small fp32 tensors, as when an adapter or a probe is trained: latency
        dict(name="norm tiny f32", op="norm", param="f32", grad="f32", pad=64, scale=1, **tiny),
        # fp16 training with a loss scale; odd sizes, every tensor starting at an odd element
        dict(name="norm odd f16 unaligned", op="norm", param="f16", grad="f16", pad=1, scale=65536, **odd),
        # the largest model of the range, gradients in bf16
        dict(name="norm large bf16", op="norm", param="bf16", grad="bf16", pad=64, scale=1, **big),
        # the same small list, stepped
        dict(name="adamw32 tiny f32", op="adamw", state=32, param="f32", grad="f32", pad=64, scale=1, step=1, skip=0, **tiny),
        # fp16 with its loss scale, odd and unaligned
        dict(name="adamw32 odd f16 unaligned", op="adamw", state=32, param="f16", grad="f16", pad=1, scale=65536, step=77, skip=0, **odd),
        # bf16 params with fp32 accumulated gradients
        dict(name="adamw32 large bf16", op="adamw", state=32, param="bf16", grad="f32", pad=64, scale=1, step=2000, skip=0, **big),
        # 8-bit moments: the small list, odd sizes (blocks that end inside), fp32 params, and the largest
        dict(name="adamw8 tiny bf16", op="adamw", state=8, param="bf16", grad="bf16", pad=256, scale=1, step=3, skip=0, **tiny),
        dict(name="adamw8 odd f16", op="adamw", state=8, param="f16", grad="f16", pad=256, scale=65536, step=900, skip=0, **odd),
        dict(name="adamw8 mid f32", op="adamw", state=8, param="f32", grad="f32", pad=256, scale=1, step=40, skip=0,
             layers=16, d=1024, ffn=2816, vocab=50000),
        dict(name="adamw8 large bf16", op="adamw", state=8, param="bf16", grad="bf16", pad=256, scale=1, step=5000, skip=0, **big),
        # moments of a running fp32 optimizer taken over into 8 bits
        dict(name="pack odd f32", op="pack", param="f32", values="f32", pad=256, **odd),
        # and back, for a checkpoint in fp32
        dict(name="unpack large f32", op="unpack", param="f32", values="f32", pad=256, **big),
    ]


def draw(rng):
    op = rng.choice(["norm", "adamw", "adamw", "adamw8", "adamw8", "pack", "unpack"])
    n = math.exp(rng.uniform(math.log(2e4), math.log(1.2e9)))
    layers = int(round(math.exp(rng.uniform(0, math.log(32)))))
    r = math.exp(rng.uniform(math.log(0.2), math.log(30)))  # vocab / d
    f = rng.uniform(1.0, 4.0)                               # ffn / d
    d = max(5, int(math.sqrt(n / ((4 + 3 * f) * layers + 2 * r))))
    size = dict(layers=layers, d=d, ffn=max(3, int(f * d)), vocab=max(2, int(r * d)))
    size = {k: v + (v == 3 * 1024) for k, v in size.items()}
    param = rng.choice(["bf16", "f16", "f32"])
    grad = param if rng.random() < 0.6 else "f32"
    scale = 65536 if grad == "f16" else rng.choice([1, 1, 8])
    if op == "norm":
        return dict(op="norm", param=param, grad=grad, pad=rng.choice([1, 3, 64]), scale=scale, **size)
    if op.startswith("adamw"):
        return dict(op="adamw", state=8 if op == "adamw8" else 32, param=param, grad=grad,
                    pad=256 if op == "adamw8" else rng.choice([1, 8, 64]), scale=scale,
                    step=rng.randint(1, 20000), skip=int(rng.random() < 0.1), **size)
    return dict(op=op, param="f32", values=rng.choice(["f32", "bf16"]), pad=256, **size)


# ------------------------------------------------------------------ sizes --

def tensors_of(case):
    """(elements, is a matrix) of each tensor, in the model's order."""
    L, d, f, v = case["layers"], case["d"], case["ffn"], case["vocab"]
    layer = [(d * d, True)] * 4 + [(f * d, True)] * 3 + [(d, False)] * 2
    return [(v * d, True)] + layer * L + [(d, False), (v * d, True)]


def groups_of(case):
    """The flat buffers: matrices, then vectors; each a list of (start, elements, place in the model's order)."""
    out = []
    for matrix in (True, False):
        at, places = 0, []
        for k, (n, is_matrix) in enumerate(tensors_of(case)):
            if is_matrix == matrix:
                at = -(-at // case["pad"]) * case["pad"]
                places.append((at, n, k))
                at += n
        unit = math.lcm(case["pad"], 8)
        out.append(dict(matrix=matrix, places=places, total=-(-at // unit) * unit,
                        param=case["param"] if matrix else "f32",
                        grad=case.get("grad", "f32") if matrix else "f32"))
    return out


def work(case):
    n_m = sum(n for n, matrix in tensors_of(case) if matrix)
    n_v = sum(n for n, matrix in tensors_of(case) if not matrix)
    if case["op"] == "norm":
        return {"bytes": n_m * SIZE[case["grad"]] + n_v * 4, "flops": 2 * (n_m + n_v)}
    if case["op"] == "adamw":
        # gradient; the fp32 weight in and out; the 16-bit param out; the moments in and out, and, of 8 bits, out as bf16 values
        state = 16 if case["state"] == 32 else 2 * 2 + 4 / BLOCK + 4
        per_m = SIZE[case["grad"]] + 8 + (2 if case["param"] != "f32" else 0) + state
        return {"bytes": n_m * per_m + n_v * (4 + 8 + state), "flops": 16 * (n_m + n_v)}
    codes, values = 2 + 2 / BLOCK, 2 * SIZE[case["values"]]
    per = values + codes + (4 if case["op"] == "pack" else 0)  # packed moments also come back as bf16 values
    return {"bytes": (n_m + n_v) * per, "flops": 4 * (n_m + n_v)}


# ----------------------------------------------------- the 8-bit encoding --
# Blocks of 256 elements.  m: e4m3 times a power of two.  v: the top bits of the fp32 pattern above the block's
# base, 5 of the exponent and 3 of the mantissa; 0 is zero.  A block that is not finite has the scale byte 255.

def encode_m(m):
    b = m.view(-1, BLOCK)
    top = ((b.abs().amax(1).view(torch.int32).long() + 0x1FFFFF) >> 23)
    scale = torch.where(top >= 255, 255, (top - 8).clamp(min=8))
    up = torch.where(top >= 255, 0, (254 - scale) << 23).to(torch.int32).view(torch.float32)
    q = torch.where((top >= 255)[:, None], 0.0, b * up[:, None]).to(torch.float8_e4m3fn)
    return q.view(torch.uint8).view(-1), scale.to(torch.uint8)


def decode_m(codes, scale):
    unit = torch.where(scale == 255, 0x7FC00000, scale.int() << 23).to(torch.int32).view(torch.float32)
    return (codes.view(torch.float8_e4m3fn).view(-1, BLOCK).float() * unit[:, None]).view(-1)


def encode_v(v, r20):
    b = v.view(-1, BLOCK)
    bits = b.view(torch.int32)
    top = (bits.amax(1).long() + 0xFFFFF) >> 23
    scale = torch.where(top >= 255, 255, (top - 31).clamp(min=0))
    c = (bits + r20 - (scale << 23).to(torch.int32)[:, None]) >> 20
    c = torch.where(bits > 0, c.clamp(1, 255), 0)
    return torch.where((top >= 255)[:, None], 0, c).to(torch.uint8).view(-1), scale.to(torch.uint8)


def decode_v(codes, scale):
    c = codes.view(-1, BLOCK).int()
    bits = torch.where(c > 0, (c << 20) + (scale.int() << 23)[:, None], 0)
    return torch.where((scale == 255)[:, None], 0x7FC00000, bits).to(torch.int32).view(torch.float32).view(-1)


def rounding_bits(block_index, ordinal, step):
    """20-bit rounding addends of every element of every block: 16 hashed bits, two elements to a hash."""
    pair = block_index[:, None] * (BLOCK // 2) + torch.arange(BLOCK // 2, device=block_index.device)[None]
    key = (SEED + ordinal * 0x510E527F + step * 0x6A09E667) & M32
    x = (pair * 0x9E3779B9 + key[:, None]) & M32
    x = x * 0xBB67AE85
    x = (x ^ (x >> 32)) & M32
    x = x * 0xA54FF53B
    x = (x ^ (x >> 32)) & M32
    return torch.stack((x & 0xFFFF, x >> 16), 2).view(-1, BLOCK).to(torch.int32) << 4


# ----------------------------------------------------------------- inputs --

def prepare(case, seed):
    dev = torch.device("cuda")
    gen = torch.Generator(dev)
    gen.manual_seed(seed)

    def normal(n):
        return torch.randn(n, generator=gen, device=dev)

    st = dict(case=dict(case), groups=[], inv=1.0 / case.get("scale", 1), t=case.get("step", 1))
    for g in groups_of(case):
        n = g["total"]
        keep = torch.zeros(n, dtype=torch.bool, device=dev)
        for at, m, _ in g["places"]:
            keep[at:at + m] = True
        if g["matrix"]:  # rows of the first matrix (the embedding) that no token of the batch touched
            keep[: g["places"][0][1] // 8] = False
        q = dict(g)
        size = normal(n).mul_(0.7).exp_().mul_(1e-3).mul_(keep)  # each element's usual gradient
        if case["op"] in ("norm", "adamw"):
            q["grad_buf"] = normal(n).mul_(size).mul_(float(case["scale"])).to(DT[g["grad"]])
        if case["op"] != "norm":
            m = normal(n).mul_(size).mul_(0.3)
            v = torch.rand(n, generator=gen, device=dev).add_(0.5).mul_(size).mul_(size)
        del size
        if case["op"] == "adamw":
            w = normal(n).mul_(0.02)
            for (at, k, _), nxt in zip(g["places"], [p[0] for p in g["places"][1:]] + [n]):
                w[at + k:nxt] = 0.0
            q["weight"] = w
            q["param_buf"] = w.to(DT[g["param"]]) if g["param"] != "f32" else w
        if case["op"] in ("pack", "unpack") or case.get("state") == 8:
            index = np.concatenate([np.arange(-(-k // BLOCK)) for _, k, _ in g["places"]])
            order = np.concatenate([np.full(-(-k // BLOCK), o) for _, k, o in g["places"]])
            q["block_index"], q["ordinal"] = torch.from_numpy(index).to(dev), torch.from_numpy(order).to(dev)
        if case["op"] == "unpack" or case.get("state") == 8:
            q["m"], q["m_scale"] = encode_m(m)
            q["v"], q["v_scale"] = encode_v(v, 0x80000)
        elif case["op"] == "pack":
            q["m_val"], q["v_val"] = m.to(DT[case["values"]]), v.to(DT[case["values"]])
            q["m"], q["v"] = (torch.zeros(n, dtype=torch.uint8, device=dev) for _ in range(2))
            q["m_scale"], q["v_scale"] = (torch.zeros(n // BLOCK, dtype=torch.uint8, device=dev) for _ in range(2))
        elif case["op"] == "adamw":
            q["m"], q["v"] = m, v
        if case["op"] in ("pack", "unpack") or case.get("state") == 8:
            out = DT[case["values"]] if case["op"] == "unpack" else torch.bfloat16
            q["m_out"], q["v_out"] = (torch.zeros(n, dtype=out, device=dev) for _ in range(2))
        st["groups"].append(q)
    st["coef"] = torch.rand(1, generator=gen, device=dev).mul_(0.5).add_(0.5)
    st["found"] = torch.full((1,), int(case.get("skip", 0)), dtype=torch.int32, device=dev)
    if own:
        _own_handles(st)
    return st


def _views(q, name):
    """Each tensor's view of flat buffer `name` (one value per element, or one per block)."""
    if q[name].numel() == q["total"]:
        return [q[name][at:at + k] for at, k, _ in q["places"]]
    return [q[name][at // BLOCK:at // BLOCK + -(-k // BLOCK)] for at, k, _ in q["places"]]


def _own_handles(st):
    """The tensor lists, marshalled once, and the workspace, as a training program keeps them."""
    import mixed_precision_adam_gb300 as dopt
    case = st["case"]
    entries = {}
    for q in st["groups"]:
        names = [k for k in ("grad_buf", "param_buf", "weight", "m", "v", "m_scale", "v_scale", "m_val", "v_val", "m_out", "v_out") if k in q]
        views = {k: _views(q, k) for k in names}
        for j, (_, _, k) in enumerate(q["places"]):
            entries[k] = (q, {name: v[j] for name, v in views.items()})
    ordered = [entries[k] for k in range(len(entries))]
    if case["op"] == "norm":
        st["list"] = dopt.TensorList([dict(grad=e["grad_buf"]) for _, e in ordered])
        st["ws"] = torch.zeros(dopt.dopt_tensors_workspace_bytes(len(ordered)), dtype=torch.uint8, device="cuda")
        st["out"] = (torch.zeros(1, device="cuda"), torch.zeros(1, device="cuda"),
                     torch.zeros(1, dtype=torch.int32, device="cuda"))
    if case["op"] == "adamw":
        small = dict(exp_avg_scale="m_scale", exp_avg_sq_scale="v_scale") if case["state"] == 8 else {}
        st["list"] = dopt.TensorList([
            dict(param=e["param_buf"], grad=e["grad_buf"], master=e["weight"] if q["param"] != "f32" else None,
                 exp_avg=e["m"], exp_avg_sq=e["v"], wd_mult=1.0 if q["matrix"] else 0.0,
                 **{k: e[v] for k, v in small.items()}) for q, e in ordered])
        st["hp"] = dict(lr=LR, beta1=B1, beta2=B2, eps=EPS, weight_decay=WD)
    if "m_out" in st["groups"][0]:
        def moments(m, v):
            return dopt.MomentList([dict(exp_avg=e[m], exp_avg_sq=e[v], exp_avg_codes=e["m"], exp_avg_sq_codes=e["v"],
                                         exp_avg_scale=e["m_scale"], exp_avg_sq_scale=e["v_scale"]) for _, e in ordered])
        st["out_list"] = moments("m_out", "v_out")
        if case["op"] == "pack":
            st["in_list"] = moments("m_val", "v_val")


# -------------------------------------------------------------------- run --

def run(state):
    case = state["case"]
    if own:
        return _run_own(state)
    if case["op"] == "norm":
        return _norm(state)
    if case["op"] == "adamw":
        return {"matrices" if q["matrix"] else "vectors": _adamw(state, q) for q in state["groups"]}
    return {"matrices" if q["matrix"] else "vectors": _pack(q) if case["op"] == "pack" else _unpack(q, DT[case["values"]])
            for q in state["groups"]}


def _run_own(st):
    import mixed_precision_adam_gb300 as dopt
    case = st["case"]
    stream = torch.cuda.current_stream()
    if case["op"] == "norm":
        norm, coef, found = st["out"]
        dopt.dopt_tensors_grad_norm(st["list"], st["inv"], MAX_NORM, st["ws"], st["ws"].numel(), norm, coef, found, stream=stream)
        return dict(norm=norm, coef=coef, found=found)
    if case["op"] == "adamw":
        dopt.dopt_tensors_adam_step(st["list"], st["hp"], st["t"], st["inv"], SEED, st["coef"], st["found"], stream=stream)
    if case["op"] == "pack":
        dopt.dopt_state8_pack(st["in_list"], stream=stream)
    if "out_list" in st:
        dopt.dopt_state8_unpack(st["out_list"], stream=stream)
    return {"matrices" if q["matrix"] else "vectors": _outputs(st["case"], q) for q in st["groups"]}


def _outputs(case, q):
    out = {}
    if case["op"] == "adamw":
        out["param"] = q["param_buf"]
        if q["param"] != "f32":
            out["master"] = q["weight"]
    eight = "m_out" in q
    out["exp_avg"], out["exp_avg_sq"] = (q["m_out"], q["v_out"]) if eight else (q["m"], q["v"])
    return out


def _norm(st):
    gs = [q["grad_buf"].float() * st["inv"] for q in st["groups"]]
    sumsq = sum((g * g).sum() for g in gs)
    found = ~(torch.isfinite(gs[0]).all() & torch.isfinite(gs[1]).all())
    norm = torch.sqrt(sumsq)
    coef = MAX_NORM / (norm + 1e-6)
    coef = torch.where(coef < 1, coef, 1.0)
    return dict(norm=torch.where(found, math.nan, norm).view(1), coef=coef.view(1), found=found.int().view(1))


def _adamw(st, q):
    case, skip = st["case"], st["found"].bool()
    eight = case["state"] == 8
    m, v = (decode_m(q["m"], q["m_scale"]), decode_v(q["v"], q["v_scale"])) if eight else (q["m"], q["v"])
    g = (q["grad_buf"].float() * st["inv"]) * st["coef"]
    w = q["weight"] * float(1.0 - LR * WD * (1.0 if q["matrix"] else 0.0))
    m1 = m * B1 + g * (1.0 - B1)
    v1 = v * B2 + (g * (1.0 - B2)) * g
    del g
    denom = torch.sqrt(v1) / math.sqrt(1.0 - B2 ** st["t"]) + EPS
    w = w - (m1 / denom) * (LR / (1.0 - B1 ** st["t"]))
    del denom
    q["weight"].copy_(torch.where(skip, q["weight"], w))
    if q["param"] != "f32":
        q["param_buf"].copy_(torch.where(skip, q["param_buf"], w.to(DT[q["param"]])))
    del w
    if not eight:
        q["m"].copy_(torch.where(skip, q["m"], m1))
        q["v"].copy_(torch.where(skip, q["v"], v1))
        return _outputs(case, q)
    r20 = rounding_bits(q["block_index"], q["ordinal"], st["t"])
    new = encode_m(m1) + encode_v(v1, r20)
    del r20, m1, v1
    q["m"].copy_(torch.where(skip, q["m"], new[0]))
    q["m_scale"].copy_(torch.where(skip, q["m_scale"], new[1]))
    q["v"].copy_(torch.where(skip, q["v"], new[2]))
    q["v_scale"].copy_(torch.where(skip, q["v_scale"], new[3]))
    return dict(_outputs(case, q), **_unpack(q, torch.bfloat16))


def _pack(q):
    q["m"], q["m_scale"] = encode_m(q["m_val"].float())
    q["v"], q["v_scale"] = encode_v(q["v_val"].float(), 0x80000)
    return _unpack(q, torch.bfloat16)


def _unpack(q, dtype):
    return dict(exp_avg=decode_m(q["m"], q["m_scale"]).to(dtype), exp_avg_sq=decode_v(q["v"], q["v_scale"]).to(dtype))


# ------------------------------------------------------------------ exact --

def exact(case, seed):
    st = prepare(case, seed)
    if case["op"] == "norm":
        # tensor by tensor, the squares' sum in 64 bits
        total, bad = 0.0, False
        for q in st["groups"]:
            for at, n, _ in q["places"]:
                x = q["grad_buf"][at:at + n].double().div_(case["scale"])
                bad = bad or not bool(torch.isfinite(x).all())
                total += float(torch.dot(x, x))
        norm = math.sqrt(total) if not math.isnan(total) else math.nan
        ratio = MAX_NORM / (norm + 1e-6)
        f = lambda x: torch.tensor([x], dtype=torch.float64)  # noqa: E731
        return dict(norm=f(math.nan if bad else norm), coef=f(ratio if ratio < 1 else 1.0),
                    found=torch.tensor([int(bad)], dtype=torch.int32))
    out = {}
    for q in st["groups"]:
        flat = {}

        def put(name, at, x):
            if name not in flat:
                flat[name] = torch.zeros(q["total"], dtype=torch.float64, device=x.device)
            flat[name][at:at + x.numel()] = x

        for at, n, k in q["places"]:
            blocks = slice(at // BLOCK, at // BLOCK + -(-n // BLOCK))
            if case["op"] == "pack":
                m, v = q["m_val"][at:at + n].double(), q["v_val"][at:at + n].double()
                put("exp_avg", at, _exact_m(m))
                put("exp_avg_sq", at, _exact_v(v, 0.5))
                continue
            if case["op"] == "unpack" or case["state"] == 8:
                m, v = _exact_values(q["m"][at:at + n], q["m_scale"][blocks], q["v"][at:at + n], q["v_scale"][blocks])
            else:
                m, v = q["m"][at:at + n].double(), q["v"][at:at + n].double()
            if case["op"] == "adamw":
                w = q["weight"][at:at + n].double()
                p = q["param_buf"][at:at + n].double()
                if not case["skip"]:
                    g = q["grad_buf"][at:at + n].double() / case["scale"] * float(st["coef"])
                    m = B1 * m + (1 - B1) * g
                    v = B2 * v + (1 - B2) * g.square()
                    w = w * (1 - LR * WD * q["matrix"]) \
                        - LR * (m / (1 - B1 ** st["t"])) / ((v / (1 - B2 ** st["t"])).sqrt() + EPS)
                    p = w
                    if case["state"] == 8:
                        m, v = _exact_m(m), _exact_v(v, _exact_fraction(n, k, st["t"], v.device))
                put("param", at, p)
                if q["param"] != "f32":
                    put("master", at, w)
            put("exp_avg", at, m)
            put("exp_avg_sq", at, v)
        out["matrices" if q["matrix"] else "vectors"] = flat
    return out


def _times2(x, e):
    """x times 2 to the whole power e, exactly."""
    return x * ((e.long() + 1023) << 52).view(torch.float64)


def _rows(x):
    """x in rows of a block, the last one filled up with zeros."""
    full = torch.zeros(-(-x.numel() // BLOCK) * BLOCK, dtype=x.dtype, device=x.device)
    full[: x.numel()] = x
    return full.view(-1, BLOCK)


def _exact_values(mc, ms, vc, vs):
    """What codes stand for, from their bit fields."""
    a = mc.long()
    e, f = (a >> 3) & 15, (a & 7).double()
    mag = torch.where(e > 0, _times2(1 + f / 8, e - 7), _times2(f / 8, torch.full_like(e, -6)))
    m = _times2(torch.where(a >= 128, -mag, mag), ms.long().repeat_interleave(BLOCK)[: a.numel()] - 127)
    c = vc.long()
    top = (c >> 3) + vs.long().repeat_interleave(BLOCK)[: c.numel()]
    f = (c & 7).double()
    v = torch.where(top > 0, _times2(1 + f / 8, top - 127), _times2(f / 8, torch.full_like(top, -126)))
    return m, torch.where(c > 0, v, torch.zeros_like(v))


def _exact_m(m):
    """Nearest multiples of the block's step: 3 bits below the leading one, and no finer than 2^-9 of the block's unit."""
    r = _rows(m)
    fr, ex = torch.frexp(r.abs().amax(1))
    unit = (ex - 1 + (fr * 2 > 1.75).int() - 8).clamp(min=8 - 127)  # the largest is in (224, 448] of the unit
    _, e = torch.frexp(r)
    step = torch.maximum(e - 4, (unit - 9)[:, None])
    return _times2(_times2(r, -step).round(), step).view(-1)[: m.numel()]


def _exact_v(v, fraction):
    """Between the two nearest values with 3 bits below the leading one: up where the fraction says so."""
    r = _rows(v)
    fr, ex = torch.frexp(r.amax(1))
    low = (ex - 1 + (fr * 2 > 1.875).int() - 31).clamp(min=-127)
    _, e = torch.frexp(r)
    step = e - 4
    u = _rows(fraction) if torch.is_tensor(fraction) else fraction
    x = _times2(torch.floor(_times2(r, -step) + u), step)
    least = _times2(torch.full_like(r[:, :1], 1.125), low[:, None])
    return torch.where(r > 0, torch.maximum(x, least), x).view(-1)[: v.numel()]


def _exact_fraction(n, ordinal, step, device):
    j = torch.arange(n, device=device)
    x = ((j >> 1) * 0x9E3779B9 + ((SEED + ordinal * 0x510E527F + step * 0x6A09E667) % 2**32)) % 2**32
    for c in (0xBB67AE85, 0xA54FF53B):
        lo, hi = (x & 0xFFFF) * c, (x >> 16) * c  # the 64-bit product from two of 48 bits
        low = (lo + ((hi & 0xFFFF) << 16)) & M32
        high = ((lo >> 16) + hi) >> 16
        x = low ^ (high & M32)
    return torch.where(j % 2 == 0, x & 0xFFFF, x >> 16).double() / 65536
