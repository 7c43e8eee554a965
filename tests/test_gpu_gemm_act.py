"""GPU parity of the FP8 products with bias, activation and residual in their
epilogue, against float64.

Tolerance.  The sum's error E is the plain products' (see test_gpu_gemm.py):
(K - 1) u sum|a b| + 3 u (|y| + |bias|), u = 2^-24.  An activation passes it on
with a slope of at most 1.13 (gelu; silu 1.1, relu 1) and adds its own: the
hardware exponential and quotient and erfc are within a few ulp of their
arguments, and an argument z of the exponential (of erfc: z^2 / 2) rounded
once moves the result by z u; results vanish below |z| = 104, so 2^-15
relative covers it, and 2^-126 what underflows.  The residual's sum rounds
once more, and the output to half a bf16 step (2^-8).
"""
import math

import pytest
import torch

pytestmark = pytest.mark.gpu
U = 2.0 ** -24
SMS = 148  # B200
ACTS = ("none", "relu", "gelu", "gelu_tanh", "silu")


@pytest.fixture(scope="module")
def rrf():
    import reduce_rmsnorm_fp8_b200 as m
    m.rrf_device_error(clear=True)
    yield m
    assert m.rrf_device_error() == 0


def randn(g, *shape):
    return torch.randn(shape, generator=g, device="cuda")


def problem(rrf, seed, m, n, k, mx=False, bias=True, residual=True, spread=1.0):
    """Operands whose products spread over +-`spread` and more."""
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    p = dict(mx=mx, m=m, n=n, k=k)
    for name, rows, size in (("a", m, 1.0), ("b", n, spread / math.sqrt(k))):
        x = randn(g, rows, k)
        p[name] = x.clamp(-4, 4).mul(100).to(torch.float8_e4m3fn)
        if mx:
            code = torch.randint(118, 123, (rows, k // 32), generator=g, device="cuda").byte()
            p["s" + name] = rrf.mx_blocked(code)
            scale = torch.exp2(code.double() - 127).repeat_interleave(32, dim=1)
            if name == "b":  # the product's size by the scales
                code.sub_(max(0, round(math.log2(math.sqrt(k) / spread))))
                p["sb"] = rrf.mx_blocked(code)
                scale = torch.exp2(code.double() - 127).repeat_interleave(32, dim=1)
        else:
            s = (0.5 + torch.rand(rows, generator=g, device="cuda")) * size / 100
            p["s" + name] = s
            scale = s.double()[:, None]
        p[name + "d"] = p[name].double() * scale
    p["bias"] = randn(g, n).bfloat16() if bias else None
    p["residual"] = randn(g, m, n).bfloat16() if residual else None
    return p


def activate(y, act):
    """float64, without cancellation below 0."""
    if act == "relu":
        return y.clamp(min=0)
    if act == "silu":
        return y / (1 + torch.exp(-y))
    if act == "gelu":
        return 0.5 * y * torch.special.erfc(-y * math.sqrt(0.5))
    if act == "gelu_tanh":
        return y / (1 + torch.exp(-2 * math.sqrt(2 / math.pi) * (y + 0.044715 * y ** 3)))
    return y


def call(rrf, p, act, rows=None, **kw):
    f = rrf.rrf_scaled_mm_mxfp8_act if p["mx"] else rrf.rrf_scaled_mm_fp8_act
    return f(p["a"], p["sa"], p["b"], p["sb"], bias=p["bias"], activation=act,
             residual=p["residual"], **kw)


def check(p, got, act, residual, label=""):
    rows = slice(None) if p["m"] <= 512 else torch.tensor(
        sorted({0, 1, 127, 128, 255, 256, p["m"] // 2, p["m"] - 2, p["m"] - 1}), device="cuda")
    ad = p["ad"][rows]
    y, mag = ad @ p["bd"].T, ad.abs() @ p["bd"].abs().T
    bias = 0.0 if p["bias"] is None else p["bias"].double()
    err = (p["k"] - 1) * U * mag + 3 * U * (y.abs() + abs(bias))
    z = activate(y + bias, act)
    err = 1.13 * err + z.abs() * 2.0 ** -15 + 2.0 ** -126
    if residual is not None:
        z = z + residual[rows].double()
        err = err + U * (z.abs() + err)
    tol = err + 2.0 ** -8 * (z.abs() + err) + 2.0 ** -134
    worst = float(((got[rows].double() - z).abs() / tol).max())
    assert worst <= 1.0, f"{label} {act}: {worst:.3f} of the bound"


# every kernel of the planner (kernel, A rows, columns; a split kernel's CTAs to
# a tile), per row / column scales and MX
FP8 = [(1, 256, 128, "swap", 8, 64), (9, 528, 640, "swap", 16, 64),
       (24, 336, 384, "swap", 32, 64), (3, 320, 1152, "swap", 8, 64),
       (32, 7168, 512, "swap", 32, 64), (5, 256, 144, "tile", 64, 64),
       (64, 5120, 1024, "tile", 64, 64), (37, 272, 256, "tile", 64, 64),
       (50, 16400, 1024, "tile", 64, 128), (130, 400, 144, "tile", 128, 64),
       (200, 272, 384, "tile", 128, 64), (250, 7184, 272, "tile", 128, 128),
       (800, 2320, 2048, "tile", 128, 128), (500, 7168, 2048, "pair", 256, 256),
       (2000, 2576, 8208, "pair", 256, 256), (4096, 8192, 1040, "pair", 256, 256),
       (24, 336, 1536, "split", 32, 2), (31, 2064, 7168, "split", 32, 2),
       (1, 2000, 4224, "split", 32, 4), (8, 912, 4224, "split", 32, 8),
       (64, 4624, 1664, "split", 64, 2), (40, 1040, 3200, "split", 64, 4),
       (33, 272, 7168, "split", 64, 8), (100, 4624, 2048, "split", 128, 2),
       (250, 784, 3456, "split", 128, 4), (129, 336, 4352, "split", 128, 8),
       # K % 128 != 0 behind boxes of several k-tiles
       (64, 5120, 528, "tile", 64, 64), (37, 272, 272, "tile", 64, 64),
       (3, 7184, 1040, "tile", 64, 64), (50, 16400, 1136, "tile", 64, 128),
       (200, 272, 400, "tile", 128, 64), (100, 4112, 656, "tile", 128, 64),
       (24, 336, 1552, "split", 32, 4), (40, 1040, 3216, "split", 64, 4),
       (8, 912, 4240, "split", 32, 8), (129, 336, 4368, "split", 128, 8),
       (100, 4624, 2064, "split", 128, 2)]
MX = [(1, 256, 128, "swap", 8, 64), (16, 208, 512, "swap", 16, 64),
      (29, 7168, 1664, "swap", 32, 64), (60, 1040, 384, "tile", 64, 64),
      (33, 16400, 640, "tile", 64, 128), (200, 272, 384, "tile", 128, 64),
      (800, 2320, 1024, "tile", 128, 128), (500, 7168, 2048, "pair", 256, 256),
      (2000, 8208, 2176, "pair", 256, 256),
      (20, 4624, 1536, "split", 32, 2), (2, 2000, 2176, "split", 32, 4),
      (32, 912, 4224, "split", 32, 8), (64, 4624, 1664, "split", 64, 2),
      (40, 1104, 3200, "split", 64, 4), (33, 336, 7168, "split", 64, 8),
      (100, 4624, 2048, "split", 128, 2), (250, 784, 3456, "split", 128, 4),
      (129, 336, 4352, "split", 128, 8)]


@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("m,n,k,kernel,rows,columns,mx",
                         [(*s, False) for s in FP8] + [(*s, True) for s in MX])
def test_matches_float64(rrf, m, n, k, kernel, rows, columns, mx, act):
    plan = rrf.rrf_plan_scaled_mm_act(m, n, k, SMS, mx=mx)
    last = plan["ctas"] // plan["tiles"] if kernel == "split" else plan["tile_n"]
    assert (plan["kernel"], plan["a_rows"], last) == (kernel, rows, columns), plan
    for bias, residual in ((True, True), (False, True), (True, False), (False, False)):
        p = problem(rrf, m + n + k, m, n, k, mx, bias, residual, spread=2.0)
        check(p, call(rrf, p, act), act, p["residual"], f"bias {bias} residual {residual}")


@pytest.mark.parametrize("m", [1, 5, 33, 64, 70, 200])
@pytest.mark.parametrize("n,k,mx", [(16, 128, False), (32, 144, False), (48, 16, False),
                                    (16, 128, True), (80, 256, True)])
def test_narrow_products(rrf, m, n, k, mx):
    """Fewer columns than a tile, a chunk or a box."""
    p = problem(rrf, m + n, m, n, k, mx)
    guard = torch.full((m * n + 128,), 7.0, dtype=torch.bfloat16, device="cuda")
    out = guard[64:64 + m * n].view(m, n)
    check(p, call(rrf, p, "gelu", out=out), "gelu", p["residual"])
    assert bool((guard[:64] == 7).all()) and bool((guard[64 + m * n:] == 7).all())


@pytest.mark.parametrize("m", [3, 40, 100, 600])
def test_scales_and_bias_of_any_alignment(rrf, m):
    """The row and column scales need 4 bytes, the bias 2."""
    p = problem(rrf, m, m, 2576, 256)
    want = call(rrf, p, "silu")
    for name in ("sa", "sb", "bias"):
        x = p[name]
        wide = torch.zeros(x.numel() + 1, dtype=x.dtype, device="cuda")
        wide[1:] = x
        p[name] = wide[1:]
        assert p[name].data_ptr() % 16 == x.element_size()
    assert torch.equal(call(rrf, p, "silu"), want)


@pytest.mark.parametrize("m,n,k,mx", [(8, 16384, 1024, False), (1, 9488, 128, False),
                                      (12, 18960, 128, True), (24, 16384, 4096, False),
                                      (40, 18960, 4096, False), (24, 18960, 4096, True),
                                      (64, 37888, 1024, False), (50, 37888, 1024, True),
                                      (70, 18960, 256, True), (70, 18960, 128, False),
                                      (2048, 2576, 1040, False), (700, 9488, 128, True),
                                      (4096, 4096, 512, False),
                                      (4096, 4096, 512, True), (4096, 4096, 2048, False),
                                      (4096, 4096, 2048, True)])
def test_several_tiles_of_a_block(rrf, m, n, k, mx):
    plan = rrf.rrf_plan_scaled_mm_act(m, n, k, SMS, mx=mx)
    assert plan["tiles"] > plan["ctas"] // (2 if plan["kernel"] == "pair" else 1), plan
    p = problem(rrf, m, m, n, k, mx)
    check(p, call(rrf, p, "silu"), "silu", p["residual"])


@pytest.mark.parametrize("m,k,mx", [(1, 256, False), (20, 256, True), (60, 256, False),
                                    (300, 256, False), (3000, 256, True), (3000, 256, False),
                                    (7, 4096, False), (60, 4096, True), (100, 4096, False)])
def test_residual_in_place(rrf, m, k, mx):
    p = problem(rrf, 7, m, 2064, k, mx)
    keep = p["residual"].clone()
    out = call(rrf, p, "gelu", out=p["residual"])
    assert out.data_ptr() == p["residual"].data_ptr()
    check(p, out, "gelu", keep)


@pytest.mark.parametrize("mx", [False, True])
def test_without_epilogue_it_is_the_plain_product(rrf, mx):
    for m in (1, 40, 150, 2048):
        p = problem(rrf, m, m, 2048, 256, mx, residual=False)
        plain = rrf.rrf_scaled_mm_mxfp8 if mx else rrf.rrf_scaled_mm_fp8
        want = plain(p["a"], p["sa"], p["b"], p["sb"], p["bias"])
        assert torch.equal(call(rrf, p, "none"), want)
        # and a zero residual adds nothing but the sign of a zero
        p["residual"] = torch.zeros_like(want)
        assert torch.equal(call(rrf, p, "none"), want)


@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("m", [4, 200])
def test_far_values_of_the_activations(rrf, act, m):
    """Sums from -1e30 to 1e30, each product one value: exact, so the error is
    the activation's alone.  One side ends at 0 or keeps the value."""
    n = k = 128
    far = torch.tensor([0.0, 1e-30, 1e-4, 0.5, 3.0, 6.0, 9.0, 12.0, 30.0, 60.0, 88.0, 103.0,
                        1e3, 1e10, 1e15, 1e30])
    value = torch.cat((far, -far)).repeat(n // 32).cuda()
    p = dict(mx=False, m=m, n=n, k=k, bias=None, residual=None,
             a=torch.zeros((m, k), device="cuda"), b=torch.eye(n, device="cuda"),
             sa=torch.ones(m, device="cuda"), sb=value)
    p["a"][:, :] = 1.0
    p["a"], p["b"] = (p[x].to(torch.float8_e4m3fn) for x in "ab")
    got = call(rrf, p, act).double()
    z = activate(value.double(), act)[None]
    tol = z.abs() * (2.0 ** -15 + 2.0 ** -8) + 2.0 ** -126
    assert not bool(got.isnan().any())
    assert bool(((got - z).abs() <= tol).all())


def test_infinities_and_nan_stay_in_their_place(rrf):
    for m in (4, 40, 300, 2048):
        p = problem(rrf, m, m, 2048, 256)
        want = call(rrf, p, "silu")
        p["residual"][1, 5] = float("nan")
        p["residual"][2, 6] = float("inf")
        got = call(rrf, p, "silu")
        assert bool(got[1, 5].isnan()) and float(got[2, 6]) == float("inf")
        got[1, 5], got[2, 6] = want[1, 5], want[2, 6]
        assert torch.equal(got, want)


def test_captured_and_on_another_stream(rrf):
    p = problem(rrf, 3, 33, 1040, 384)
    out = torch.empty((33, 1040), dtype=torch.bfloat16, device="cuda")
    call(rrf, p, "gelu_tanh", out=out)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call(rrf, p, "gelu_tanh", out=out)
    p["residual"].neg_()
    out.zero_()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        graph.replay()
    side.synchronize()
    check(p, out, "gelu_tanh", p["residual"])


def test_a_block_of_projections(rrf):
    """The fused call's codes through an up projection with its activation,
    and back down into the residual it wrote, in place."""
    import parity
    import workloads
    c = parity.to_device(workloads.make_case("decode", 32, cols=1024))
    q, s, h = rrf.rrf_sum_rmsnorm_fp8(c.inputs, c.gamma, c.eps, c.weight_offset, c.scale_ub,
                                      residual_in=c.residual.clone())
    up = problem(rrf, 1, 32, 2048, 1024, residual=False)
    up.update(a=q, sa=s.reshape(-1), ad=q.double() * s.double())
    mid = call(rrf, up, "silu")
    check(up, mid, "silu", None, "up")
    # the activations quantised by the same call (gamma 1)
    one = torch.ones(2048, dtype=torch.bfloat16, device="cuda")
    q2, s2, _ = rrf.rrf_sum_rmsnorm_fp8([mid], one, 1e-6, 0.0, float("inf"))
    down = problem(rrf, 2, 32, 1024, 2048)
    keep = h.clone()
    down.update(a=q2, sa=s2.reshape(-1), ad=q2.double() * s2.double(), residual=h)
    out = call(rrf, down, "none", out=h)
    check(down, out, "none", keep, "down")


def test_refusals_of_tensors(rrf):
    p = problem(rrf, 1, 8, 64, 128)
    args = (p["a"], p["sa"], p["b"], p["sb"])
    f = rrf.rrf_scaled_mm_fp8_act
    for bad in (dict(activation="tanh"), dict(residual=p["residual"][:4]),
                dict(residual=p["residual"].float()), dict(residual=p["residual"].T),
                dict(out=torch.empty((8, 64), device="cuda")), dict(bias=p["bias"][:10]),
                dict(residual=p["residual"].cpu())):
        with pytest.raises(ValueError):
            f(*args, **bad)
    with pytest.raises(rrf.RrfError) as e:  # a residual that only partly is out
        buf = torch.empty(9 * 64, dtype=torch.bfloat16, device="cuda")
        f(*args, residual=buf[:512].view(8, 64), out=buf[64:].view(8, 64))
    assert e.value.status == rrf.Status.ERR_ALIAS


@pytest.mark.parametrize("m,n,k,mx", [(4, 1024, 4096, False), (60, 1024, 4096, True),
                                      (200, 7168, 1024, False), (600, 7168, 2048, False)])
def test_wait_timeout_is_reported(rrf, m, n, k, mx):
    """The test hook makes a bounded wait of the epilogue run out: the call ends,
    reports it, and the next call is right.  Two calls of a split product give
    the same bits."""
    p = problem(rrf, 5, m, n, k, mx)
    torch.cuda.synchronize()
    rrf.rrf_debug_starve_next_gemm()
    call(rrf, p, "silu")
    torch.cuda.synchronize()
    assert rrf.rrf_device_error(clear=True) & rrf.RRF_DEVICE_ERROR_GEMM_TIMEOUT
    out = call(rrf, p, "silu")
    check(p, out, "silu", p["residual"])
    assert torch.equal(out, call(rrf, p, "silu"))


@pytest.mark.parametrize("m,n,k", [(5, 4096, 128), (14, 2048, 256), (30, 2048, 128), (40, 2048, 384),
                                   (40, 2048, 144), (200, 1024, 256), (1000, 2576, 128),
                                   (3000, 2576, 256), (1, 1024, 4224), (64, 1024, 4096),
                                   (250, 784, 3456)])
def test_scales_and_bias_round_one_by_one(rrf, m, n, k):
    """((sum * a_scale) * b_scale) + bias, each step rounded to fp32: bit for
    bit, in the plain product and in the one with an epilogue.  The sums are
    small integers (exact in fp32 in any order), and the bias takes most of the
    first row away, so that a step left unrounded shows in one value of some
    hundred."""
    g = torch.Generator(device="cuda")
    g.manual_seed(m + n)
    a, b = (torch.randint(-2, 4, (rows, k), generator=g, device="cuda").float().to(
        torch.float8_e4m3fn) for rows in (m, n))
    sums = (a.double() @ b.double().T).float()
    sa = 0.5 + torch.rand(m, generator=g, device="cuda") / 64
    sb = 0.5 + torch.rand(n, generator=g, device="cuda")
    y = (sums * sa[:, None]) * sb
    bias = -y[0].bfloat16()
    want = (y + bias.float()).bfloat16()
    assert torch.equal(rrf.rrf_scaled_mm_fp8(a, sa, b, sb, bias), want)
    assert torch.equal(rrf.rrf_scaled_mm_fp8_act(a, sa, b, sb, bias), want)
    # (the case can tell: with one rounding fewer some values differ)
    once = (sums.double() * sa.double()[:, None]).float().double() * sb.double() + bias.double()
    assert bool((once.float().bfloat16() != want).any())


@pytest.mark.parametrize("m,n,k,kernel,mx", [
    (4, 1024, 4096, "split", False), (60, 1024, 4096, "split", True),
    (64, 4624, 1664, "split", False), (129, 336, 4352, "split", False),
    (100, 4624, 2048, "split", True), (4, 7168, 512, "swap", False), (4, 7168, 512, "swap", True),
    (64, 5120, 528, "tile", False), (200, 7168, 1024, "tile", False),
    (200, 7168, 1024, "tile", True), (500, 7168, 2048, "pair", False),
    (500, 7168, 2048, "pair", True)])
def test_a_wait_that_ran_out_stores_nothing(rrf, m, n, k, kernel, mx):
    """An output tile whose sums did not come is left as it was."""
    assert rrf.rrf_plan_scaled_mm_act(m, n, k, SMS, mx=mx)["kernel"] == kernel
    p = problem(rrf, 6, m, n, k, mx)
    out = torch.full((m, n), 7.0, dtype=torch.bfloat16, device="cuda")
    torch.cuda.synchronize()
    rrf.rrf_debug_starve_next_gemm()
    call(rrf, p, "silu", out=out)
    torch.cuda.synchronize()
    assert rrf.rrf_device_error(clear=True) & rrf.RRF_DEVICE_ERROR_GEMM_TIMEOUT
    assert bool((out == 7).all())
    check(p, call(rrf, p, "silu", out=out), "silu", p["residual"])


# small cases of every kernel of the planner, with a last stage of fewer bytes
# (K % 128 != 0) where there is one
CHECKED = [(5, 256, 128, "swap", 8, False), (14, 272, 256, "swap", 16, False),
           (30, 336, 384, "swap", 32, False), (5, 256, 144, "tile", 64, False),
           (64, 5120, 528, "tile", 64, False), (50, 16400, 1136, "tile", 64, False),
           (37, 272, 112, "tile", 64, False),
           (200, 272, 112, "tile", 128, False), (200, 272, 400, "tile", 128, False),
           (250, 7184, 272, "tile", 128, False), (700, 9488, 128, "pair", 256, False),
           (24, 336, 1552, "split", 32, False), (8, 912, 4240, "split", 32, False),
           (40, 1040, 3216, "split", 64, False), (129, 336, 4368, "split", 128, False),
           (1, 256, 128, "swap", 8, True), (16, 208, 512, "swap", 16, True),
           (29, 336, 384, "swap", 32, True), (60, 1040, 384, "tile", 64, True),
           (33, 16400, 640, "tile", 64, True), (200, 272, 384, "tile", 128, True),
           (250, 7184, 256, "tile", 128, True), (700, 9488, 128, "pair", 256, True),
           (20, 4624, 1536, "split", 32, True), (40, 1104, 3200, "split", 64, True),
           (129, 336, 4352, "split", 128, True)]

_CHECKED = r'''
import sys
sys.path[:0] = [ROOT, HERE]
import reduce_rmsnorm_fp8_b200 as rrf
import test_gpu_gemm_act as t
assert rrf.LIB_PATH.endswith("librrf_debug.so"), rrf.LIB_PATH
rrf.rrf_device_error(clear=True)
for m, n, k, kernel, rows, mx in t.CHECKED:
    p = t.problem(rrf, m + n, m, n, k, mx)
    t.check(p, t.call(rrf, p, "gelu"), "gelu", p["residual"], "residual")
    keep = p["residual"].clone()
    t.check(p, t.call(rrf, p, "silu", out=p["residual"]), "silu", keep, "in place")
    p["residual"] = None
    t.check(p, t.call(rrf, p, "none"), "none", None, "no residual")
    plain = rrf.rrf_scaled_mm_mxfp8 if mx else rrf.rrf_scaled_mm_fp8
    t.check(p, plain(p["a"], p["sa"], p["b"], p["sb"], p["bias"]), "none", None, "plain")
assert rrf.rrf_device_error() == 0, rrf.rrf_device_error()
print("checked build clean")
'''


def test_bounds_checking_build(rrf):
    """Every kernel of the planner in the bounds-checking build: right, with a
    clear error word."""
    import os
    import subprocess
    import sys
    from reduce_rmsnorm_fp8_b200 import build
    for m, n, k, kernel, rows, mx in CHECKED:
        plan = rrf.rrf_plan_scaled_mm_act(m, n, k, SMS, mx=mx)
        assert (plan["kernel"], plan["a_rows"]) == (kernel, rows), (m, n, k, mx, plan)
    build.build(debug=True)
    here = os.path.dirname(os.path.abspath(__file__))
    root = os.path.dirname(here)
    p = subprocess.run([sys.executable, "-c", f"ROOT = {root!r}\nHERE = {here!r}\n" + _CHECKED],
                       env=dict(os.environ, RRF_DEBUG_LIBRARY="1"), cwd=root,
                       capture_output=True, text=True, timeout=600)
    assert p.returncode == 0 and "checked build clean" in p.stdout, (p.stdout + p.stderr)[-4000:]


def check_all(p, got, act, residual, label=""):
    """check() on every row, 512 at a time."""
    for r in range(0, p["m"], 512):
        rows = slice(r, min(r + 512, p["m"]))
        part = {**p, "m": rows.stop - r, "ad": p["ad"][rows]}
        check(part, got[rows], act, None if residual is None else residual[rows],
              f"{label} rows {r}..")


@pytest.mark.parametrize("m,n,k,kernel,columns,mx", [
    (2000, 2576, 8208, "pair", 256, False), (4096, 8192, 1040, "pair", 256, False),
    (4096, 4096, 2048, "pair", 256, False), (4096, 4096, 2048, "pair", 256, True),
    (2000, 8208, 2176, "pair", 256, True), (4096, 4096, 512, "tile", 128, True),
    (3000, 2064, 256, "tile", 128, False), (3000, 2064, 256, "tile", 128, True),
    (4096, 4096, 512, "tile", 128, False), (1999, 2576, 1024, "tile", 128, True),
    (700, 9488, 128, "pair", 256, True), (700, 9488, 128, "pair", 256, False)])
def test_every_row(rrf, m, n, k, kernel, columns, mx):
    """Every row of the products whose blocks take several tiles: each warp's
    box and barrier in turn, both accumulators; with and without a residual,
    in place, and the plain product, which has the same epilogue."""
    plan = rrf.rrf_plan_scaled_mm_act(m, n, k, SMS, mx=mx)
    assert (plan["kernel"], plan["tile_n"]) == (kernel, columns), plan
    assert plan["tiles"] > plan["ctas"] // (2 if kernel == "pair" else 1), plan
    p = problem(rrf, m + k, m, n, k, mx)
    keep = p["residual"]
    check_all(p, call(rrf, p, "gelu"), "gelu", keep, "residual")
    p["residual"] = keep.clone()
    out = call(rrf, p, "silu", out=p["residual"])
    check_all(p, out, "silu", keep, "in place")
    p["residual"] = None
    check_all(p, call(rrf, p, "relu"), "relu", None, "no residual")
    plain = rrf.rrf_scaled_mm_mxfp8 if mx else rrf.rrf_scaled_mm_fp8
    check_all(p, plain(p["a"], p["sa"], p["b"], p["sb"], p["bias"]), "none", None, "plain")


def test_written_outputs_count_a_version(rrf):
    for mx in (False, True):
        p = problem(rrf, 2, 4, 64, 128, mx)
        for out in (torch.empty_like(p["residual"]), p["residual"]):
            before = out._version
            call(rrf, p, "silu", out=out)
            assert out._version > before
