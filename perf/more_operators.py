"""Training in 8 bits next to the optimizer step: what is computed, on what sizes.

Four operators:

  pack     a matrix to e4m3 codes with one power-of-two scale per 128 columns
           of a row ("row") or per 128 x 128 square ("square"), and its
           transpose likewise; both returned as the values the codes stand for
  product  D = A B^T of two such matrices, stored or added to D
  norm     root-mean-square norm of the rows of h = dropout(x) + residual,
           returned as values or, in 8 bits, as the values the codes stand
           for; and its backward pass
  dropout  from a counter-based generator, the residual added

The scale bytes of a matrix lie in the order the matrix unit reads them:
128 rows by 4 blocks in 512 bytes (scale_offsets).
"""

import math

import torch

own = False

BLOCK = 128
DT = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
SIZE = {"f32": 4, "bf16": 2, "f16": 2}
EPS = 1e-6
SEED, SITE, STEP = 1234567, 3, 41  # of the dropout
M32 = 0xFFFFFFFF


def listed():
    return [
        # a handful of tokens through a feed-forward matrix, as when a trained model is sampled: latency
        dict(name="product 16 tokens", op="product", rows=16, cols=5504, depth=2048, out="bf16", add=0, pad=0, square=1),
        # odd sizes, into a slice of wider rows, in fp32
        dict(name="product odd f32", op="product", rows=1001, cols=769, depth=2051, out="f32", add=0, pad=13, square=0),
        # the forward pass of a feed-forward matrix of the 7B shape, eight sequences of 2048
        dict(name="product large bf16", op="product", rows=16384, cols=11008, depth=4096, out="bf16", add=0, pad=0, square=1),
        # the same matrix's gradient, added to the fp32 grad that the optimizer step reads
        dict(name="product weight grad f32", op="product", rows=11008, cols=4096, depth=16384, out="f32", add=1, pad=0, square=0),
        # the norm before a product, a handful of tokens
        dict(name="norm 8 tokens", op="norm", rows=8, cols=2048, dtype="bf16", residual=1, p=0.0, eight=1),
        # and sixteen sequences of 2048
        dict(name="norm large bf16 to 8 bits", op="norm", rows=32768, cols=4096, dtype="bf16", residual=1, p=0.0, eight=1),
        # the backward pass, odd sizes in fp16 with dropout on the branch
        dict(name="norm backward odd f16", op="norm_back", rows=4099, cols=769, dtype="f16", residual=1, p=0.1),
        # and the large one
        dict(name="norm backward large bf16", op="norm_back", rows=32768, cols=4096, dtype="bf16", residual=1, p=0.0),
        # gradients of odd sizes to 8 bits, for the two products of the backward pass
        dict(name="pack odd bf16", op="pack", rows=4099, cols=2051, dtype="bf16", block="row", both=1),
        # the fp32 weights of a feed-forward matrix after a step, for the forward and the backward pass
        dict(name="pack weights f32", op="pack", rows=11008, cols=4096, dtype="f32", block="square", both=1),
        # dropout of a small activation: latency
        dict(name="dropout small bf16", op="dropout", rows=128, cols=768, dtype="bf16", residual=0, p=0.1),
        # of sixteen sequences of 2048, added to the residual
        dict(name="dropout large bf16", op="dropout", rows=32768, cols=4096, dtype="bf16", residual=1, p=0.1),
    ]


def _spread(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["product", "product", "norm", "norm", "norm_back", "norm_back", "pack", "dropout"])
    odd = rng.random() < 0.5
    if op == "product":
        rows, cols, depth = _spread(rng, 1, 16384), _spread(rng, 64, 12000), _spread(rng, 64, 8192)
        if not odd:
            cols, depth = -(-cols // 128) * 128, -(-depth // 128) * 128
        rows = max(1, min(rows, 738000000000 // (cols * depth)))  # of the largest listed product
        add = int(rng.random() < 0.3)
        out = "f32" if add else rng.choice(["f32", "bf16", "bf16", "f16"])
        return dict(op=op, rows=rows, cols=cols, depth=depth, out=out, add=add,
                    pad=rng.choice([0, 0, 1, 8, 64]), square=rng.randint(0, 1))
    rows, cols = _spread(rng, 1, 30000), _spread(rng, 96, 8192)
    if not odd:
        cols = -(-cols // 64) * 64
    rows = max(1, min(rows, 130000000 // cols))
    dtype = rng.choice(["bf16", "bf16", "f16", "f32"])
    if op == "pack":
        return dict(op=op, rows=min(rows, 45000000 // cols), cols=cols, dtype=dtype, block=rng.choice(["row", "square"]), both=rng.randint(0, 1))
    p = rng.choice([0.0, 0.1, 0.25])
    if op == "dropout":
        return dict(op=op, rows=rows, cols=cols, dtype=dtype, residual=rng.randint(0, 1), p=max(p, 0.05))
    if op == "norm":
        return dict(op=op, rows=rows, cols=cols, dtype=dtype, residual=rng.randint(0, 1), p=p, eight=rng.randint(0, 1))
    return dict(op=op, rows=rows, cols=cols, dtype=dtype, residual=rng.randint(0, 1), p=p)


def work(case):
    r, c = case["rows"], case["cols"]
    if case["op"] == "product":
        k = case["depth"]
        blocks = -(-k // BLOCK)
        return {"bytes": (r + c) * (k + blocks) + r * c * SIZE[case["out"]] * (2 if case["add"] else 1), "flops": 2 * r * c * k}
    n, size = r * c, SIZE[case["dtype"]]
    if case["op"] == "pack":  # values in; per orientation the codes out, and them as bf16 values
        scales = r * c / BLOCK if case["block"] == "row" else r * c / BLOCK ** 2
        return {"bytes": n * size + (1 + case["both"]) * (n * 3 + scales), "flops": 2 * (1 + case["both"]) * n}
    if case["op"] == "dropout":
        return {"bytes": n * size * (2 + case["residual"]), "flops": 4 * n}
    if case["op"] == "norm":
        stored = case["residual"] or case["p"] > 0  # h is another array than x
        out = 3 + 1 / BLOCK if case["eight"] else size  # codes, and them as bf16 values
        return {"bytes": n * (size * (1 + case["residual"] + stored) + out) + 4 * (c + r), "flops": 6 * n}
    return {"bytes": n * size * (3 + case["residual"] + (case["p"] > 0)) + 4 * (3 * c + r), "flops": 10 * n}


# ------------------------------------------------------------- the encoding --

def scale_offsets(rows, blocks, device):
    """Place of the scale byte of each row and block."""
    r = torch.arange(rows, device=device)[:, None]
    b = torch.arange(blocks, device=device)[None]
    return ((r // 128) * -(-blocks // 4) + b // 4) * 512 + (r % 32) * 16 + (r % 128) // 32 * 4 + b % 4


def scale_bytes(rows, cols):
    return -(-rows // 128) * -(-cols // 512) * 512


def encode(x, square):
    """Codes (uint8) and the scale of each row and block, of fp32 values."""
    rows, cols = x.shape
    blocks = -(-cols // BLOCK)
    x = torch.nn.functional.pad(x, (0, blocks * BLOCK - cols)) if blocks * BLOCK > cols else x
    x = x.reshape(rows, blocks, BLOCK)
    top = x.abs().amax(2)
    if square:
        tall = -(-rows // BLOCK)
        top = torch.nn.functional.pad(top, (0, 0, 0, tall * BLOCK - rows)).view(tall, BLOCK, blocks).amax(1)
        top = top.repeat_interleave(BLOCK, 0)[:rows]
    e = (top.contiguous().view(torch.int32).long() + 0x1FFFFF) >> 23
    scale = torch.where(e >= 255, 255, (e - 8).clamp(min=8))
    up = torch.where(e >= 255, 0, (254 - scale) << 23).to(torch.int32).view(torch.float32)
    codes = torch.where((e >= 255)[..., None], 0.0, x * up[..., None]).to(torch.float8_e4m3fn)
    return codes.view(torch.uint8).view(rows, -1)[:, :cols], scale.to(torch.uint8)


def decode(codes, scale):
    """fp32 values of codes, from the scale of each row and block."""
    unit = torch.where(scale == 255, 0x7FC00000, scale.int() << 23).to(torch.int32).view(torch.float32)
    return codes.view(torch.float8_e4m3fn).float() * unit.repeat_interleave(BLOCK, 1)[:, : codes.shape[1]]


def stored(codes, scale):
    """A matrix as it is kept: rows of codes on 16-byte boundaries, scales in the matrix unit's order."""
    rows, cols = codes.shape
    kept = torch.zeros(rows, -(-cols // 16) * 16, dtype=torch.uint8, device=codes.device)[:, :cols]
    kept.copy_(codes)
    scales = torch.zeros(scale_bytes(rows, cols), dtype=torch.uint8, device=codes.device)
    scales[scale_offsets(rows, scale.shape[1], codes.device)] = scale
    return kept, scales


def values_of(codes, scales):
    """fp32 values of a matrix as it is kept."""
    rows, cols = codes.shape
    return decode(codes.contiguous(), scales[scale_offsets(rows, -(-cols // BLOCK), codes.device)])


def threshold(p):
    return int(round(p * 65536))


def kept_mask(rows, cols, p, device):
    """Which elements stay: 16 hashed bits per element, two elements to a hash."""
    n = rows * cols
    x = (torch.arange((n + 1) // 2, device=device) * 0x9E3779B9 + SEED + SITE * 0x510E527F + STEP * 0x6A09E667) & M32
    x = x * 0xBB67AE85
    x = (x ^ (x >> 32)) & M32
    x = x * 0xA54FF53B
    x = (x ^ (x >> 32)) & M32
    r = torch.stack((x & 0xFFFF, x >> 16), 1).view(-1)[:n]
    return (r >= threshold(p)).view(rows, cols)


def dropped(x, p):
    """fp32 values after the dropout."""
    if p == 0:
        return x
    return torch.where(kept_mask(*x.shape, p, x.device), x * (65536 / (65536 - threshold(p))), 0.0)


# ------------------------------------------------------------------- inputs --

def prepare(case, seed):
    dev = torch.device("cuda")
    gen = torch.Generator(dev)
    gen.manual_seed(seed)

    def normal(*shape):
        return torch.randn(*shape, generator=gen, device=dev)

    def activations(rows, cols):  # a few columns are many times larger, as a trained model's are
        x = normal(rows, cols)
        return x.mul_(normal(cols).mul_(0.7).exp_())

    def gradients(rows, cols):  # rows (tokens) of very different size
        x = normal(rows, cols)
        return x.mul_(normal(rows, 1).exp_().mul_(1e-3))

    r, c = case["rows"], case["cols"]
    st = dict(case=dict(case))
    if case["op"] == "product":
        k = case["depth"]
        if case["add"]:  # both operands transposed: tokens along the rows
            st["a"] = stored(*encode(gradients(k, r).t().contiguous(), False))
            st["b"] = stored(*encode(activations(k, c).t().contiguous(), case["square"]))
        else:
            st["a"] = stored(*encode(activations(r, k), False))
            st["b"] = stored(*encode(normal(c, k).mul_(0.02), case["square"]))
        st["d"] = torch.zeros(r, c + case["pad"], dtype=DT[case["out"]], device=dev)[:, :c]
        if case["add"]:
            st["d"].copy_(normal(r, c).mul_(1e-2))
    elif case["op"] == "pack":
        x = normal(r, c).mul_(0.02) if case["block"] == "square" else gradients(r, c)
        st["x"] = x.to(DT[case["dtype"]])
        for name, (rows, cols) in (("out", (r, c)), ("out_t", (c, r)))[: 1 + case["both"]]:
            st[name] = stored(torch.zeros(rows, cols, dtype=torch.uint8, device=dev),
                              torch.zeros(rows, -(-cols // BLOCK), dtype=torch.uint8, device=dev))
            st[name + "_values"] = torch.empty(rows, cols, dtype=torch.bfloat16, device=dev)
    elif case["op"] == "dropout":
        st["x"] = activations(r, c).to(DT[case["dtype"]])
        st["residual"] = activations(r, c).to(DT[case["dtype"]]) if case["residual"] else None
        st["y"] = torch.empty_like(st["x"])
    else:
        t = DT[case["dtype"]]
        st["gain"] = normal(c).mul_(0.2).add_(1.0)
        if case["op"] == "norm":
            st["x"] = activations(r, c).to(t)
            st["residual"] = activations(r, c).mul_(2).to(t) if case["residual"] else None
            st["h"] = torch.empty_like(st["x"]) if case["residual"] or case["p"] > 0 else None
            st["rstd"] = torch.empty(r, device=dev)
            if case["eight"]:
                st["out"] = stored(torch.zeros(r, c, dtype=torch.uint8, device=dev),
                                   torch.zeros(r, -(-c // BLOCK), dtype=torch.uint8, device=dev))
                st["out_values"] = torch.empty(r, c, dtype=torch.bfloat16, device=dev)
            else:
                st["y"] = torch.empty_like(st["x"])
        else:
            st["h"] = activations(r, c).mul_(2).to(t)
            st["rstd"] = torch.rsqrt(st["h"].float().square().mean(1) + EPS)
            # fp16 gradients carry the loss scale
            st["dy"] = gradients(r, c).mul_(1024 if t == torch.float16 else 1).to(t)
            st["dres"] = gradients(r, c).mul_(1024 if t == torch.float16 else 1).to(t) if case["residual"] else None
            st["dh"] = torch.empty_like(st["h"])
            st["dx"] = torch.empty_like(st["h"]) if case["p"] > 0 else None
            st["dgain"] = normal(c).mul_(1e-2)
    if own:
        _own_handles(st)
    return st


def _own_handles(st):
    """The arguments, marshalled once, and the workspace, as a training program keeps them."""
    import mixed_precision_adam_gb300 as dopt
    case = st["case"]
    r, c = case["rows"], case["cols"]
    drop = dopt.Dropout(case["p"], SEED, site=SITE, step=STEP) if case.get("p") else None
    if case["op"] == "product":
        st["args"] = dopt.Matrix8(*st["a"]), dopt.Matrix8(*st["b"])
    elif case["op"] == "pack":
        block = dopt.BLOCK_SQUARE if case["block"] == "square" else dopt.BLOCK_ROW
        out = {k: dopt.Matrix8(*st[k]) for k in ("out", "out_t") if k in st}
        st["args"] = dopt.MatrixList([dict(values=st["x"], block=block, **out)])
        st["values"] = dopt.MatrixList([dict(values=st[k + "_values"], out=m) for k, m in out.items()])
    elif case["op"] == "dropout":
        st["args"] = dopt.DropoutArgs(st["x"], st["y"], drop, residual=st["residual"])
    elif case["op"] == "norm":
        out = dict(y8=dopt.Matrix8(*st["out"])) if case["eight"] else dict(y=st["y"])
        st["args"] = dopt.RmsNormArgs(st["x"], st["gain"], EPS, residual=st["residual"], dropout=drop, h=st["h"], rstd=st["rstd"], **out)
        if case["eight"]:
            st["values"] = dopt.MatrixList([dict(values=st["out_values"], out=out["y8"])])
    else:
        size = dopt.dopt_rms_norm_workspace_bytes(r, c)
        st["ws"] = torch.empty(size, dtype=torch.uint8, device="cuda")
        st["args"] = dopt.RmsNormBackwardArgs(st["dy"], st["h"], st["gain"], st["rstd"], st["dh"], dres=st["dres"], dropout=drop, dx=st["dx"],
                                              dgain=st["dgain"], accumulate=True, workspace=st["ws"], workspace_bytes=size)


# ---------------------------------------------------------------------- run --

def run(state):
    return _run_own(state) if own else _run_plain(state)


def _run_own(st):
    import mixed_precision_adam_gb300 as dopt
    case = st["case"]
    stream = torch.cuda.current_stream()
    if case["op"] == "product":
        dopt.dopt_matrix8_multiply(*st["args"], st["d"], accumulate=bool(case["add"]), stream=stream)
        return st["d"]
    if case["op"] == "pack":
        dopt.dopt_matrix8_pack(st["args"], stream=stream)
        dopt.dopt_matrix8_unpack(st["values"], stream=stream)
        return {k: st[k + "_values"] for k in ("out", "out_t") if k in st}
    if case["op"] == "dropout":
        dopt.dopt_dropout(st["args"], stream=stream)
        return st["y"]
    if case["op"] == "norm":
        dopt.dopt_rms_norm(st["args"], stream=stream)
        if case["eight"]:
            dopt.dopt_matrix8_unpack(st["values"], stream=stream)
        return dict(h=st["h"], rstd=st["rstd"], y=st["out_values"] if case["eight"] else st["y"])
    dopt.dopt_rms_norm_backward(st["args"], stream=stream)
    return dict(dh=st["dh"], dx=st["dx"], dgain=st["dgain"])


def _run_plain(st):
    case = st["case"]
    if case["op"] == "product":
        d = values_of(*st["a"]) @ values_of(*st["b"]).t()
        st["d"].copy_(st["d"].float() + d if case["add"] else d)
        return st["d"]
    if case["op"] == "pack":
        square, x = case["block"] == "square", st["x"].float()
        return {k: decode(*encode(x if k == "out" else x.t().contiguous(), square)).to(torch.bfloat16) for k in ("out", "out_t") if k in st}
    if case["op"] == "dropout":
        y = dropped(st["x"].float(), case["p"])
        return (y + st["residual"].float() if case["residual"] else y).to(DT[case["dtype"]])
    if case["op"] == "norm":
        h = dropped(st["x"].float(), case["p"])
        h = (h + st["residual"].float() if case["residual"] else h).to(DT[case["dtype"]])
        f = h.float()
        rstd = torch.rsqrt((f * f).mean(1) + EPS)
        y = f * rstd[:, None] * st["gain"]
        y = decode(*encode(y, False)).to(torch.bfloat16) if case["eight"] else y.to(h.dtype)
        return dict(h=h if st["h"] is not None else None, rstd=rstd, y=y)
    dy, h, rstd = st["dy"].float(), st["h"].float(), st["rstd"][:, None]
    g, hat = dy * st["gain"], h * rstd
    dh = (g - hat * (g * hat).mean(1, keepdim=True)) * rstd
    if case["residual"]:
        dh = dh + st["dres"].float()
    st["dgain"] += (dy * hat).sum(0)
    dx = dropped(dh, case["p"]).to(DT[case["dtype"]]) if case["p"] else None
    return dict(dh=dh.to(DT[case["dtype"]]), dx=dx, dgain=st["dgain"])


# -------------------------------------------------------------------- exact --

def exact(case, seed):
    st = prepare(case, seed)
    if case["op"] == "product":
        a, b = _exact_values(*st["a"]), _exact_values(*st["b"])
        d = a @ b.t()
        return d + st["d"].double() if case["add"] else d
    if case["op"] == "pack":
        x = st["x"].double()
        out = {}
        for name, v in (("out", x), ("out_t", x.t()))[: 1 + case["both"]]:
            out[name] = _exact_rounded(v, BLOCK if case["block"] == "square" else 1)
        return out
    if case["op"] == "dropout":
        y = _exact_dropped(st["x"].double(), case["p"])
        return y + st["residual"].double() if case["residual"] else y
    if case["op"] == "norm":
        h = _exact_dropped(st["x"].double(), case["p"])
        if case["residual"]:
            h = h + st["residual"].double()
        h = h.to(DT[case["dtype"]]).double()
        rstd = (h.square().sum(1) / case["cols"] + EPS).pow(-0.5)
        y = st["gain"].double() * (h * rstd[:, None])
        return dict(h=h if st["h"] is not None else None, rstd=rstd, y=_exact_rounded(y, 1) if case["eight"] else y)
    dy, h, rstd = st["dy"].double(), st["h"].double(), st["rstd"].double()[:, None]
    dgain = st["dgain"].double() + torch.einsum("rc,rc->c", dy, h * rstd)
    dot = torch.einsum("rc,rc,c->r", dy, h, st["gain"].double())[:, None]
    dh = rstd * dy * st["gain"].double() - h * (dot * rstd ** 3 / case["cols"])
    if case["residual"]:
        dh = dh + st["dres"].double()
    return dict(dh=dh, dx=_exact_dropped(dh, case["p"]) if case["p"] else None, dgain=dgain)


def _times2(x, e):
    """x times 2 to the whole power e, exactly."""
    return x * ((e.long() + 1023) << 52).view(torch.float64)


def _exact_values(codes, scales):
    """What a kept matrix stands for, from the codes' bit fields."""
    rows, cols = codes.shape
    tall, wide = -(-rows // 128), -(-cols // 512)
    # 128 x 4 bytes at a time: 32 rows of 16 bytes, four rows' scales in each
    s = scales.view(tall, wide, 32, 4, 4).permute(0, 3, 2, 1, 4).reshape(tall * 128, wide * 4)[:rows].long()
    s = s.repeat_interleave(128, 1)[:, :cols]
    a = codes.long()
    e, f = (a >> 3) & 15, (a & 7).double()
    mag = torch.where(e > 0, _times2(1 + f / 8, e - 7), _times2(f / 8, torch.full_like(e, -6)))
    return _times2(torch.where(a >= 128, -mag, mag), s - 127)


def _exact_rounded(x, tall):
    """Nearest multiples of each block's step (tall x 128): 3 bits below the leading one, no finer than 2^-9 of the block's unit."""
    rows, cols = x.shape
    up, across = -(-rows // tall), -(-cols // BLOCK)
    full = torch.zeros(up * tall, across * BLOCK, dtype=torch.float64, device=x.device)
    full[:rows, :cols] = x
    b = full.view(up, tall, across, BLOCK)
    fr, ex = torch.frexp(b.abs().amax((1, 3), keepdim=True))
    unit = (ex - 1 + (fr * 2 > 1.75).int() - 8).clamp(min=8 - 127)  # the largest is in (224, 448] of the unit
    step = torch.maximum(torch.frexp(b)[1] - 4, unit - 9)
    return _times2(_times2(b, -step).round(), step).view(up * tall, -1)[:rows, :cols]


def _exact_dropped(x, p):
    if p == 0:
        return x
    j = torch.arange(x.numel(), device=x.device)
    y = ((j >> 1) * 0x9E3779B9 + ((SEED + SITE * 0x510E527F + STEP * 0x6A09E667) % 2**32)) % 2**32
    for c in (0xBB67AE85, 0xA54FF53B):
        lo, hi = (y & 0xFFFF) * c, (y >> 16) * c  # the 64-bit product from two of 48 bits
        low = (lo + ((hi & 0xFFFF) << 16)) & M32
        high = ((lo >> 16) + hi) >> 16
        y = low ^ (high & M32)
    r = torch.where(j % 2 == 0, y & 0xFFFF, y >> 16).view(x.shape)
    drop = round(p * 65536)
    return torch.where(r < drop, torch.zeros_like(x), x / (1 - drop / 65536))
