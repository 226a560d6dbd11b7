"""The step over a list of tensors on the GPU, against its 64-bit restatement
(oracle/tensors.py): the grad norm, AdamW with fp32 and 8-bit moments, their
pack and unpack, and the whole step.  Tolerances are the first-order bounds
of the fp32 operations' roundings (there); 8-bit codes must be those of a
moment within that bound."""

import math

import numpy as np
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("needs a CUDA GPU", allow_module_level=True)

import mixed_precision_adam_gb300 as dopt  # noqa: E402
from oracle import tensors as O  # noqa: E402
from tests.tensors_harness import HP, TORCH, Array, Case, check_codes  # noqa: E402

TYPES = [("f32", "f32"), ("bf16", "bf16"), ("bf16", "f32"), ("f16", "f16"), ("f16", "f32")]
SIZES = [0, 1, 2, 7, 8, 9, 31, 255, 256, 257, 2047, 2048, 2049, 8191, 8193, 100003]


def scalars():
    return torch.full((1,), -1.0, device="cuda"), torch.full((1,), -1.0, device="cuda"), \
        torch.full((1,), -1, dtype=torch.int32, device="cuda")


def run_norm(lst, inv=1.0, max_norm=1.0, stream=None):
    """(norm, coef, found, zeros) of a list; the workspace starts as noise."""
    ws = torch.randint(0, 255, (dopt.dopt_tensors_workspace_bytes(lst.n),), dtype=torch.uint8, device="cuda")
    out = scalars()
    torch.cuda.synchronize()
    dopt.dopt_tensors_grad_norm(lst, inv, max_norm, ws, ws.numel(), *out, stream=stream)
    st = dopt.dopt_read_step_stats(ws, stream)
    torch.cuda.synchronize()
    norm, coef, found = (x.item() for x in out)
    assert st["found_inf"] == found and st["kernel_error"] == 0
    assert (st["grad_norm"] == norm or math.isnan(norm)) and st["clip_coef"] == coef
    return norm, coef, found, st["num_zeros"]


# sum of n squares: at most 16 fp32 additions in a row, the square (1), the grad's scale (2, squared), 19 roundings
# on positive terms, halved by the root, and the result's own: 10.5 half ulps
NORM_RTOL = 11 * O.U


def check_norm(lst, grads, inv=1.0, max_norm=1.0):
    want = O.grad_norm(grads, inv, max_norm)
    got = run_norm(lst, inv, max_norm)
    assert got[2] == int(want[2]) and got[3] == want[3], (got, want)
    if want[2]:
        assert math.isnan(got[0])
        return got
    assert abs(got[0] - want[0]) <= NORM_RTOL * want[0], (got, want)
    assert abs(got[1] - want[1]) <= (NORM_RTOL + O.U) * want[1], (got, want)
    return got


# ------------------------------------------------------------------- norm --

@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("offset", [0, 1, 3, 8])
def test_norm_sizes_and_offsets(dtype, offset):
    gen = torch.Generator().manual_seed(5)
    arrays = [Array(torch.randn(n, generator=gen) * (torch.rand(n, generator=gen) > 0.1), TORCH[dtype], offset)
              for n in SIZES]
    for a in arrays:  # one tensor at a time, and all
        check_norm(dopt.TensorList([dict(grad=a.view)]), [a.numpy()], 0.5, 0.25)
    check_norm(dopt.TensorList([dict(grad=a.view) for a in arrays]), [a.numpy() for a in arrays], 0.5, 1e9)
    assert all(a.guards_intact() for a in arrays)


def test_norm_of_nothing():
    assert run_norm(dopt.TensorList([])) == (0.0, 1.0, 0, 0)
    empty = dict(grad=torch.zeros(0, device="cuda"))
    assert run_norm(dopt.TensorList([empty, empty])) == (0.0, 1.0, 0, 0)


@pytest.mark.parametrize("count", [63, 64, 65, 1279, 1280, 1281, 3000])
def test_norm_of_many_tensors(count):
    """Counts around what one launch's table holds."""
    gen = torch.Generator().manual_seed(count)
    flat = torch.randn(40 * count, generator=gen).cuda()
    dts = [torch.float32, torch.bfloat16, torch.float16]
    grads = [flat[40 * k: 40 * k + 1 + (k * 7) % 40].to(dts[k % 3]) for k in range(count)]
    check_norm(dopt.TensorList([dict(grad=g) for g in grads]), [g.float().cpu().numpy() for g in grads])


@pytest.mark.parametrize("bad", [math.inf, -math.inf, math.nan])
@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("n,where", [(1, 0), (9, 8), (5000, 4999), (100003, 70001)])
def test_norm_finds_one_bad_value(bad, dtype, n, where):
    g = torch.ones(n, dtype=TORCH[dtype], device="cuda")
    g[where] = bad
    got = check_norm(dopt.TensorList([dict(grad=g)]), [g.float().cpu().numpy()])
    # the coefficient follows the formula: 1 / inf is 0, and a NaN is not below 1
    assert got[1] == (1.0 if math.isnan(bad) else 0.0)


@pytest.mark.parametrize("size", [1e-42, 1e-30, 1e-20, 1e15, 3e19, 3e38])
@pytest.mark.parametrize("n", [1, 13, 30000])
def test_norm_of_extreme_values(size, n):
    """Squares beyond fp32's range on either side, alone and among ordinary values."""
    g = np.random.default_rng(3).standard_normal(n).clip(-1.1, 1.1).astype(np.float32) * np.float32(size)
    mixed = np.concatenate([g, np.ones(100, np.float32), np.zeros(50, np.float32)])
    for x in (g, mixed):
        d = torch.from_numpy(x).cuda()
        want = math.sqrt((x.astype(np.float64) ** 2).sum())
        got = run_norm(dopt.TensorList([dict(grad=d)]), 1.0, 0.0)
        assert got[2] == 0 and got[1] == 1.0 and got[3] == (x == 0).sum()
        if want > 3.4e38:
            assert got[0] == math.inf  # the norm itself is beyond fp32
        else:
            assert abs(got[0] - want) <= NORM_RTOL * want + 2.0**-150


def test_norm_overflow_by_the_unscale_is_found():
    g = torch.full((1000,), 1e30, device="cuda")
    assert run_norm(dopt.TensorList([dict(grad=g)]), 1.0)[2] == 0
    assert run_norm(dopt.TensorList([dict(grad=g)]), 1e20)[2] == 1


def test_norm_gives_the_same_bits_every_time():
    gen = torch.Generator(device="cuda").manual_seed(9)
    grads = [torch.randn(n, generator=gen, device="cuda") for n in (1000003, 17, 5000000)]
    lst = dopt.TensorList([dict(grad=g) for g in grads])
    assert len({run_norm(lst)[:2] for _ in range(20)}) == 1


# ------------------------------------------------------------------- step --

def adam(case, step, seed=0, inv=1.0, coef=None, found=None, hp=HP, stream=None):
    dopt.dopt_tensors_adam_step(case.list, hp, step, inv, seed, coef, found, stream=stream)


@pytest.mark.parametrize("types", TYPES)
@pytest.mark.parametrize("moments", [32, 8])
@pytest.mark.parametrize("offset", [0, 1, 4, 8])
def test_step_sizes_and_offsets(types, moments, offset):
    """Every size, three steps (the state carries over), one list."""
    case = Case([dict(numel=n, param=types[0], grad=types[1], moments=moments, offset=offset,
                      wd_mult=[1.0, 0.0, 0.3][k % 3], zero=0.2 * (k % 2)) for k, n in enumerate(SIZES)],
                seed=offset + moments, scale=1024.0)
    coef = torch.tensor([0.37], device="cuda")
    for step in (1, 2, 1000):
        adam(case, step, seed=99, inv=1 / 1024, coef=coef)
        case.check_step(step, 1 / 1024, float(coef), 99)


@pytest.mark.parametrize("types", [("f32", "f32"), ("bf16", "bf16"), ("f16", "f32")])
@pytest.mark.parametrize("moments", [32, 8])
@pytest.mark.parametrize("by", [1, 4, 8, 16])
def test_step_with_one_array_off_the_others_grid(types, moments, by):
    """Each array in turn starts `by` elements further on than the rest."""
    names = ["param", "grad", "exp_avg", "exp_avg_sq"] + (["master"] if types[0] != "f32" else []) + \
        (["exp_avg_scale", "exp_avg_sq_scale"] if moments == 8 else [])
    case = Case([dict(numel=n, param=types[0], grad=types[1], moments=moments, offsets={name: by})
                 for name in names for n in (5, 2500, 30000)], seed=by)
    for step in (1, 2):
        adam(case, step, seed=5)
        case.check_step(step, seed=5)


def test_step_of_a_mixed_list():
    """Every type and moment format in one list, in no order."""
    tensors = []
    for k in range(60):
        p, g = TYPES[(k * 7) % 5]
        tensors.append(dict(numel=[0, 5, 256, 1000, 3001, 70000][k % 6], param=p, grad=g, moments=[32, 8][(k // 3) % 2],
                            offset=[0, 0, 1, 32][k % 4], wd_mult=k / 60))
    case = Case(tensors, seed=4)
    for step in (5, 6):
        adam(case, step, seed=2**32 - 1)
        case.check_step(step, seed=2**32 - 1)


@pytest.mark.parametrize("count", [39, 40, 41, 399, 400, 401, 1000])
@pytest.mark.parametrize("moments", [32, 8])
def test_step_of_many_tensors(count, moments):
    """Counts around what one launch's table holds."""
    case = Case([dict(numel=1 + (k * 37) % 300, param="bf16", grad="bf16", moments=moments) for k in range(count)], seed=6)
    adam(case, 3, seed=1)
    case.check_step(3, seed=1)


@pytest.mark.parametrize("moments", [32, 8])
def test_skipped_step_writes_nothing(moments):
    case = Case([dict(numel=n, param="bf16", grad="f32", moments=moments, offset=n % 2) for n in (1000, 4097)], seed=8)
    found = torch.tensor([1], dtype=torch.int32, device="cuda")
    adam(case, 1, found=found)
    case.check_unchanged()
    found.zero_()
    adam(case, 1, found=found)
    case.check_step(1)


@pytest.mark.parametrize("hp", [dict(HP, beta1=0.0, beta2=0.0), dict(HP, lr=0.0), dict(HP, weight_decay=0.0, eps=1e-3),
                                dict(HP, beta1=0.999, beta2=0.9999)])
@pytest.mark.parametrize("moments", [32, 8])
def test_step_hyperparameters(hp, moments):
    case = Case([dict(numel=3000, param="bf16", grad="bf16", moments=moments)], seed=10)
    for step in (1, 2**31 + 5):
        adam(case, step, hp=hp)
        case.check_step(step, hp=hp)


@pytest.mark.parametrize("size", [1e-30, 1e-18, 1e10, 1e17])
def test_step8_extreme_grads(size):
    """Second moments near the ends of fp32's range, and blocks of zeros."""
    case = Case([dict(numel=5000, param="f32", grad="f32", moments=8, zero=0.5),
                 dict(numel=1024, param="f32", grad="f32", moments=8, zero=1.0)], seed=11, grad_size=size)
    for step in (1, 2, 3):
        adam(case, step)
        case.check_step(step)


def test_step8_zero_grads_keep_zero_moments():
    case = Case([dict(numel=1000, param="f32", grad="f32", moments=8, zero=1.0)], seed=12)
    adam(case, 1)
    after = case.values()[0]
    assert not after["exp_avg"].any() and not after["exp_avg_sq"].any()
    assert (after["exp_avg_scale"] == 8).all() and not after["exp_avg_sq_scale"].any()


@pytest.mark.parametrize("bad", [math.inf, math.nan])
def test_step8_bad_grad_without_a_flag_marks_its_block(bad):
    """A caller that steps a bad grad: its block reads as NaN from then on, its neighbours are untouched."""
    case = Case([dict(numel=1024, param="bf16", grad="bf16", moments=8)], seed=13)
    case.arrays[0]["grad"].view[300] = bad
    adam(case, 1)
    b = case.values()[0]
    assert list(b["exp_avg_scale"] == 255) == [False, True, False, False]
    assert list(b["exp_avg_sq_scale"] == 255) == [False, True, False, False]
    assert not b["exp_avg"][256:512].any() and not b["exp_avg_sq"][256:512].any()
    w = case.weights(b)
    assert np.flatnonzero(np.isnan(w)).tolist() == [300]
    adam(case, 2)
    w = case.weights(case.values()[0])
    assert np.isnan(w[256:512]).all() and np.isfinite(w[:256]).all() and np.isfinite(w[512:]).all()


@pytest.mark.parametrize("types", TYPES)
def test_step32_equals_the_sharded_step_bit_for_bit(types):
    """dopt_adam_step on a one-param buffer and the list's step: the same arithmetic."""
    n = 20011
    case = Case([dict(numel=n, param=types[0], grad="f32", moments=32, wd_mult=0.7)], seed=14)
    code = dict(f32=dopt.F32, bf16=dopt.BF16, f16=dopt.F16)[types[0]]
    m = dopt.dopt_build_shard_map([dict(numel=n, dtype=code, wd_mult=0.7)], 1, -1, True, False)
    info = dopt.dopt_buffer_info_get(m, 0)
    assert dopt.dopt_param_index(m, 0)[1] == 0

    def padded(x, dtype):
        out = torch.zeros(info["numel"], dtype=dtype, device="cuda")
        out[:n] = x
        return out

    a = case.arrays[0]
    main, m1, v1 = (padded(a[k].view, torch.float32) for k in ("grad", "exp_avg", "exp_avg_sq"))
    master = padded(a["master"].view, torch.float32) if "master" in a else None
    param = padded(a["param"].view, TORCH[types[0]])
    coef, found = torch.tensor([0.61], device="cuda"), torch.zeros(1, dtype=torch.int32, device="cuda")
    dopt.dopt_adam_step(m, 0, 0, main, master, m1, v1, param, HP, 17, coef, found)
    adam(case, 17, coef=coef, found=found)
    torch.cuda.synchronize()
    for got, want in ((a["exp_avg"], m1), (a["exp_avg_sq"], v1), (a["param"], param)) + \
            (((a["master"], master),) if master is not None else ()):
        assert torch.equal(got.view, want[:n])


def test_step_on_another_stream():
    """Inputs made on a side stream, the step queued right behind on it."""
    side = torch.cuda.Stream()
    case = Case([dict(numel=n, param="bf16", grad="bf16", moments=m) for n in (300007, 2000) for m in (32, 8)], seed=15)
    grads = [torch.randn(t["numel"], device="cuda").to(torch.bfloat16) * 0.01 for t in case.spec]
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        torch.cuda._sleep(20_000_000)
        for a, g in zip(case.arrays, grads):
            a["grad"].view.copy_(g)
        adam(case, 2, stream=side)
    side.synchronize()
    for b, a, g in zip(case.before, case.arrays, grads):
        b["grad"] = g.float().cpu().numpy()
    case.check_step(2)


def test_step_past_32_bit_offsets():
    """One tensor of more than 2^32 elements: windows at its start, around 2^31 and 2^32 and at its ragged end."""
    n = 2**32 + 12345
    free = torch.cuda.mem_get_info()[0]
    if free < 12 * n + (8 << 30):
        pytest.skip("not enough device memory")
    for moments in (8, 32):
        per = 4 if moments == 32 else 1
        dt = torch.float32 if moments == 32 else torch.uint8
        grad = torch.empty(n, dtype=torch.bfloat16, device="cuda").fill_(0.25)
        w = torch.empty(n, dtype=torch.float32, device="cuda").fill_(0.5)
        p = torch.empty(n, dtype=torch.bfloat16, device="cuda").fill_(0.5)
        m = torch.zeros(n, dtype=dt, device="cuda")
        v = torch.zeros(n, dtype=dt, device="cuda")
        e = dict(param=p, grad=grad, master=w, exp_avg=m, exp_avg_sq=v)
        if moments == 8:
            e["exp_avg_scale"], e["exp_avg_sq_scale"] = (torch.full((-(-n // 256),), 100, dtype=torch.uint8, device="cuda")
                                                         for _ in range(2))
        assert per * n == m.numel() * m.element_size()
        lst = dopt.TensorList([e])
        windows = [(0, 4096), (2**31 - 2048, 4096), (2**32 - 2048, 4096), (n - 5000 + (-(n - 5000)) % 256, None)]
        starts = []
        for at, size in windows:
            size = n - at if size is None else size
            g = torch.randn(size, device="cuda").to(torch.bfloat16)
            grad[at:at + size] = g
            starts.append((at, size, g.float().cpu().numpy()))
        norm, _, found, zeros = run_norm(lst)
        want = math.sqrt((n - sum(s[1] for s in starts)) * 0.0625 + sum((s[2].astype(np.float64) ** 2).sum() for s in starts))
        assert found == 0 and abs(norm - want) <= NORM_RTOL * want
        dopt.dopt_tensors_adam_step(lst, HP, 3, 1.0, 7)
        torch.cuda.synchronize()
        for at, size, g in starts:
            (w1, m1, v1), (dw, dm, dv) = O.adamw(np.full(size, 0.5), g, np.zeros(size), np.zeros(size), HP, 3)
            assert (np.abs(w[at:at + size].cpu().numpy() - w1) <= dw).all(), at
            if moments == 32:
                assert (np.abs(m[at:at + size].cpu().numpy() - m1) <= dm).all(), at
                assert (np.abs(v[at:at + size].cpu().numpy() - v1) <= dv).all(), at
            else:
                blocks = slice(at // 256, -(-(at + size) // 256))
                b = {k: e[k][at:at + size].cpu().numpy() for k in ("exp_avg", "exp_avg_sq")}
                b |= {k: e[k][blocks].cpu().numpy() for k in ("exp_avg_scale", "exp_avg_sq_scale")}
                check_codes(b, m1, dm, v1, dv, O.rounding_fraction(size, 0, 3, 7, first=at))
        del grad, w, p, m, v, e, lst
        torch.cuda.empty_cache()


def test_step8_second_moment_is_right_in_the_mean():
    """Stationary grads, beta2 = 0.999: each step moves v by about 0.1 %, far below half a code; the stochastic
    rounding keeps its mean.  The mean over 65,536 elements of the ratio to the exact moment has a standard
    error of about 0.2 / 256 (the ratio's spread, about 0.2, over the root of the count); 6 of those."""
    n, hp = 65536, dict(HP, lr=0.0, beta2=0.999, weight_decay=0.0)
    gen = torch.Generator(device="cuda").manual_seed(16)
    size = torch.exp(torch.randn(n, generator=gen, device="cuda")) * 1e-3
    grad = torch.empty(n, device="cuda")
    e = dict(param=torch.zeros(n, device="cuda"), grad=grad)
    for k in ("exp_avg", "exp_avg_sq"):
        e[k] = torch.zeros(n, dtype=torch.uint8, device="cuda")
        e[k + "_scale"] = torch.full((n // 256,), 8 if k == "exp_avg" else 0, dtype=torch.uint8, device="cuda")
    lst = dopt.TensorList([e])
    exact = torch.zeros(n, dtype=torch.float64, device="cuda")
    for t in range(1, 2001):
        torch.randn(n, generator=gen, device="cuda", out=grad)
        grad *= size
        exact = 0.999 * exact + 0.001 * grad.double() ** 2
        dopt.dopt_tensors_adam_step(lst, hp, t, 1.0, 5)
    v = O.v_values(e["exp_avg_sq"].cpu().numpy(), e["exp_avg_sq_scale"].cpu().numpy())
    ratio = v / exact.cpu().numpy()
    assert abs(ratio.mean() - 1) < 6 * 0.2 / 256, ratio.mean()
    assert ratio.std() < 0.3


# --------------------------------------------------------- pack and unpack --

def moments_case(n, dtype, offset, seed, special=False):
    gen = torch.Generator().manual_seed(seed)
    size = torch.exp(torch.randn(n, generator=gen) * 3) * 1e-4
    m, v = torch.randn(n, generator=gen) * size, torch.rand(n, generator=gen) * size * size
    if special and n > 600:
        m[:256] = 0
        v[:256] = 0
        v[300], m[301] = math.inf, math.nan
        v[600], m[600] = -0.0, -0.0
    a = dict(exp_avg=Array(m, TORCH[dtype], offset), exp_avg_sq=Array(v, TORCH[dtype], offset))
    blocks = -(-n // 256)
    for k in ("exp_avg", "exp_avg_sq"):
        a[k + "_codes"] = Array(torch.zeros(n), torch.uint8, offset)
        a[k + "_scale"] = Array(torch.zeros(blocks), torch.uint8, offset)
    return a


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("offset", [0, 1, 4, 8])
def test_pack_and_unpack(dtype, offset):
    sizes = SIZES
    cases = [moments_case(n, dtype, offset, n, special=True) for n in sizes]
    lst = dopt.MomentList([{k: x.view for k, x in a.items()} for a in cases])
    dopt.dopt_state8_pack(lst)
    torch.cuda.synchronize()
    packed = []
    for n, a in zip(sizes, cases):
        b = {k: x.numpy() for k, x in a.items()}
        m, v = b["exp_avg"].astype(np.float64), b["exp_avg_sq"].astype(np.float64)
        assert np.array_equal(b["exp_avg_scale"], O.m_scale(m)) and np.array_equal(b["exp_avg_sq_scale"], O.v_scale(v))
        mv = O.m_values(b["exp_avg_codes"], b["exp_avg_scale"])
        vv = O.v_values(b["exp_avg_sq_codes"], b["exp_avg_sq_scale"])
        assert np.array_equal(mv, O.m_rounded(m, b["exp_avg_scale"]), equal_nan=True)
        assert np.array_equal(vv, O.v_rounded(v, b["exp_avg_sq_scale"], 0.5), equal_nan=True)
        packed.append((mv, vv))
    dopt.dopt_state8_unpack(lst)
    torch.cuda.synchronize()
    for (mv, vv), a in zip(packed, cases):
        assert np.array_equal(a["exp_avg"].numpy().astype(np.float64), mv, equal_nan=True)
        assert np.array_equal(a["exp_avg_sq"].numpy().astype(np.float64), vv, equal_nan=True)
        assert all(x.guards_intact() for x in a.values())
    # packing the unpacked values again gives the same values
    dopt.dopt_state8_pack(lst)
    dopt.dopt_state8_unpack(lst)
    torch.cuda.synchronize()
    for (mv, vv), a in zip(packed, cases):
        assert np.array_equal(a["exp_avg"].numpy().astype(np.float64), mv, equal_nan=True)
        assert np.array_equal(a["exp_avg_sq"].numpy().astype(np.float64), vv, equal_nan=True)


def test_unpack_every_code():
    """Every code under scales from the smallest to the largest, in both value types."""
    scales = [0, 1, 8, 9, 100, 127, 200, 223, 246, 255]
    codes = torch.arange(256).repeat(len(scales)).to(torch.uint8)
    for dtype in ("f32", "bf16"):
        for which, values, usable in (("exp_avg", O.m_values, [s for s in scales if 8 <= s]),
                                      ("exp_avg_sq", O.v_values, [s for s in scales if s <= 223 or s == 255])):
            e = {which: torch.zeros(len(codes), dtype=TORCH[dtype], device="cuda"), which + "_codes": codes.cuda(),
                 which + "_scale": torch.tensor(scales, dtype=torch.uint8, device="cuda")}
            dopt.dopt_state8_unpack(dopt.MomentList([e]))
            got = e[which].double().cpu().numpy().reshape(-1, 256)
            with np.errstate(invalid="ignore"):
                want = values(codes.numpy(), scales).reshape(-1, 256)
            for k, s in enumerate(scales):
                if s in usable:
                    skip = np.isin(np.arange(256), [127, 255]) if which == "exp_avg" else (np.arange(256) > 0) & (s == 255)
                    assert np.array_equal(got[k][~skip], want[k][~skip], equal_nan=True), (which, dtype, s)


def test_unpack_leaves_out_what_is_not_asked_for():
    a = moments_case(1000, "f32", 0, 3)
    full = dopt.MomentList([{k: x.view for k, x in a.items()}])
    dopt.dopt_state8_pack(full)
    v0 = a["exp_avg_sq"].numpy()
    only = dopt.MomentList([dict(exp_avg=a["exp_avg"].view, exp_avg_codes=a["exp_avg_codes"].view,
                                 exp_avg_scale=a["exp_avg_scale"].view)])
    dopt.dopt_state8_unpack(only)
    torch.cuda.synchronize()
    assert np.array_equal(a["exp_avg_sq"].numpy(), v0)
    assert np.array_equal(a["exp_avg"].numpy(), O.m_values(a["exp_avg_codes"].numpy(), a["exp_avg_scale"].numpy()))


@pytest.mark.parametrize("count", [59, 60, 61, 499, 501])
def test_pack_many_tensors(count):
    cases = [moments_case(1 + k % 300, ["f32", "bf16"][k % 2], 0, k) for k in range(count)]
    dopt.dopt_state8_pack(dopt.MomentList([{k: x.view for k, x in a.items()} for a in cases]))
    torch.cuda.synchronize()
    for a in cases:
        b = {k: x.numpy() for k, x in a.items()}
        assert np.array_equal(O.m_values(b["exp_avg_codes"], b["exp_avg_scale"]),
                              O.m_rounded(b["exp_avg"].astype(np.float64), b["exp_avg_scale"]))


# ------------------------------------------------------------ whole step --

def step_list(seed):
    return Case([dict(numel=n, param=p, grad=g, moments=m) for n, (p, g), m in
                 zip((50000, 333, 7001, 4096), (TYPES[1], TYPES[0], TYPES[3], TYPES[2]), (8, 32, 8, 32))], seed=seed)


def test_whole_step_equals_its_parts():
    """dopt_tensors_step against the norm and the step called apart, and the 64-bit step; a bad grad skips it."""
    one, two = step_list(20), step_list(20)
    ws = torch.zeros(dopt.dopt_tensors_workspace_bytes(4), dtype=torch.uint8, device="cuda")
    for step in (1, 2):
        norm, coef, found = scalars()
        dopt.dopt_tensors_grad_norm(one.list, 0.5, 1e-3, ws, ws.numel(), norm, coef, found)
        adam(one, step, seed=3, inv=0.5, coef=coef, found=found)
        d_found, d_norm = scalars()[2], scalars()[0]
        dopt.dopt_tensors_step(two.list, HP, step, ws, ws.numel(), inv_loss_scale=0.5, max_norm=1e-3, seed=3,
                               d_found_inf=d_found, d_norm=d_norm)
        torch.cuda.synchronize()
        assert d_found.item() == found.item() == 0 and d_norm.item() == norm.item()
        for x, y in zip(one.values(), two.values()):
            assert all(np.array_equal(x[k], y[k]) for k in x)
        two.check_step(step, 0.5, coef.item(), 3)
    two.arrays[1]["grad"].view[5] = math.nan
    two.before = two.values()
    dopt.dopt_tensors_step(two.list, HP, 3, ws, ws.numel(), d_found_inf=d_found, d_norm=d_norm)
    torch.cuda.synchronize()
    assert d_found.item() == 1 and math.isnan(d_norm.item())
    for a, b in zip(two.before, two.values()):
        assert all(np.array_equal(a[k], b[k], equal_nan=True) for k in a)


def test_state_rewritten_by_a_kernel_right_before_each_step():
    """The AdamW launch may start under the norm's; what a kernel before the step wrote must still be what it
    reads: weights, moments and grads rewritten on the stream before every step, no wait in between."""
    live, ref = step_list(22), step_list(22)
    ws = torch.zeros(dopt.dopt_tensors_workspace_bytes(4), dtype=torch.uint8, device="cuda")
    other = step_list(23)  # other weights, moments and grads, of the same shapes
    names = ["param", "master", "grad", "exp_avg", "exp_avg_sq", "exp_avg_scale", "exp_avg_sq_scale"]
    saved = [{k: a[k].view.clone() for k in names if k in a} for a in ref.arrays]
    for step in range(1, 21):
        # live: through other values and back, on the device, right before the step
        for src in (other.arrays, saved):
            for a, b in zip(live.arrays, src):
                for k in names:
                    if k in a:
                        a[k].view.copy_(b[k].view if hasattr(b[k], "guards_intact") else b[k])
        dopt.dopt_tensors_step(live.list, HP, step, ws, ws.numel(), seed=step)
        torch.cuda.synchronize()
        for a, b in zip(ref.arrays, saved):
            for k in b:
                a[k].view.copy_(b[k])
        torch.cuda.synchronize()
        norm, coef, found = scalars()
        dopt.dopt_tensors_grad_norm(ref.list, 1.0, 1.0, ws, ws.numel(), norm, coef, found)
        torch.cuda.synchronize()
        adam(ref, step, seed=step, coef=coef, found=found)
        torch.cuda.synchronize()
        for k, (x, y) in enumerate(zip(ref.values(), live.values())):
            for name in x:
                assert np.array_equal(x[name], y[name]), (step, k, name)


def test_two_lists_on_two_streams():
    """Two lists stepped at once, each with its workspace, equal the same lists stepped alone."""
    streams = [torch.cuda.Stream() for _ in range(2)]
    cases = [step_list(30), step_list(31)]
    alone = [step_list(30), step_list(31)]
    ws = [torch.zeros(dopt.dopt_tensors_workspace_bytes(4), dtype=torch.uint8, device="cuda") for _ in range(2)]
    torch.cuda.synchronize()
    for step in range(1, 31):
        for c, w, s in zip(cases, ws, streams):
            dopt.dopt_tensors_step(c.list, HP, step, w, w.numel(), seed=9, stream=s)
    torch.cuda.synchronize()
    for c, w in zip(alone, ws):
        for step in range(1, 31):
            dopt.dopt_tensors_step(c.list, HP, step, w, w.numel(), seed=9)
        torch.cuda.synchronize()
    for c, a in zip(cases, alone):
        c.check_guards()
        for k, (x, y) in enumerate(zip(a.values(), c.values())):
            for name in x:
                assert np.array_equal(x[name], y[name]), (k, name)


def test_device_step_count_in_a_graph():
    """Captured once, replayed: the same bits as host-numbered steps; a skipped replay does not count."""
    host, dev = step_list(21), step_list(21)
    ws = torch.zeros(dopt.dopt_tensors_workspace_bytes(4), dtype=torch.uint8, device="cuda")
    count = torch.zeros(1, dtype=torch.int64, device="cuda")
    lr = torch.tensor([HP["lr"]], dtype=torch.float64, device="cuda")
    stream = torch.cuda.Stream()

    def one(s):
        dopt.dopt_tensors_step(dev.list, dict(HP, lr=123.0), 1, ws, ws.numel(), seed=4, d_step=count, d_lr=lr, stream=s)

    one(stream)  # the first step runs eagerly
    stream.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=stream):
        one(torch.cuda.current_stream())
    bad = dev.arrays[0]["grad"].view
    good = bad[7].item()
    for k in range(5):
        bad[7] = math.inf if k == 2 else good
        graph.replay()
        torch.cuda.synchronize()
    assert count.item() == 5  # 1 eager + 5 replays - 1 skipped
    ws2 = torch.zeros_like(ws)
    for step in range(1, 6):
        dopt.dopt_tensors_step(host.list, HP, step, ws2, ws2.numel(), seed=4)
    for k, (x, y) in enumerate(zip(host.values(), dev.values())):
        for name in x:
            assert np.array_equal(x[name], y[name]), (k, name)


def test_empty_list_steps():
    ws = torch.zeros(dopt.dopt_tensors_workspace_bytes(0), dtype=torch.uint8, device="cuda")
    norm = scalars()[0]
    dopt.dopt_tensors_step(dopt.TensorList([]), HP, 1, ws, ws.numel(), d_norm=norm)
    dopt.dopt_tensors_adam_step(dopt.TensorList([]), HP, 1)
    dopt.dopt_state8_pack(dopt.MomentList([]))
    torch.cuda.synchronize()
    assert norm.item() == 0.0
