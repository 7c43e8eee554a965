"""Host validation of the products with an epilogue: no GPU is touched."""
import pytest

MB = 1 << 20
M, N, K = 5, 64, 128


@pytest.fixture(scope="module")
def rrf():
    from reduce_rmsnorm_fp8_b200 import build
    build.build()
    import reduce_rmsnorm_fp8_b200 as m
    return m


CASES = [
    ({}, "OK"), (dict(residual=None, bias=None), "OK"), (dict(residual=6 * MB), "OK"),
    (dict(M=0, a=None, residual=None), "OK"), (dict(M=0, activation=9), "ERR_VALUE"),
    (dict(activation=-1), "ERR_VALUE"), (dict(activation=5), "ERR_VALUE"),
    (dict(out=None), "ERR_NULL"), (dict(sa=None), "ERR_NULL"), (dict(K=100), "ERR_SHAPE"),
    (dict(N=24), "ERR_SHAPE"), (dict(M=-1), "ERR_SHAPE"), (dict(residual=5 * MB + 8), "ERR_ALIGN"),
    (dict(bias=8 * MB + 1), "ERR_ALIGN"), (dict(out=MB), "ERR_ALIAS"),
    (dict(residual=6 * MB + 16), "ERR_ALIAS"), (dict(residual=6 * MB - 16), "ERR_ALIAS"),
    (dict(residual=6 * MB + M * N * 2), "OK"),
]


@pytest.mark.parametrize("mx", [False, True])
@pytest.mark.parametrize("change,want", CASES, ids=str)
def test_arguments(rrf, change, want, mx):
    c = dict(a=MB, sa=2 * MB, b=3 * MB, sb=4 * MB, bias=8 * MB, activation=2, residual=5 * MB,
             out=6 * MB, M=M, N=N, K=K, **{})
    c.update(change)
    f = rrf.lib.rrf_check_scaled_mm_mx_act_args if mx else rrf.lib.rrf_check_scaled_mm_act_args
    assert rrf.Status(f(*c.values())).name == want


def test_constants_match_the_header(rrf):
    import os
    import re
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    text = open(os.path.join(root, "include", "rrf.h")).read()
    for name in ("NONE", "RELU", "GELU", "GELU_TANH", "SILU"):
        assert getattr(rrf, "RRF_ACT_" + name) == \
            int(re.search(rf"#define RRF_ACT_{name} (\d+)", text).group(1))


def test_cpu_tensors_and_unknown_activations_are_refused(rrf):
    import torch
    a = torch.zeros((2, 128), dtype=torch.uint8).view(torch.float8_e4m3fn)
    s = torch.ones(2)
    with pytest.raises(ValueError):
        rrf.rrf_scaled_mm_fp8_act(a, s, a, s)


@pytest.mark.parametrize("m,n,k,mx,want", [
    (1, 7168, 7168, False, ("swap", 8, 64, 8, 112, 112)),
    (64, 16384, 7168, False, ("tile", 64, 128, 2, 128, 128)),
    (64, 7168, 7168, False, ("tile", 64, 64, 4, 112, 112)),
    (128, 7168, 4096, False, ("tile", 128, 64, 2, 112, 112)),
    (256, 7168, 4096, False, ("tile", 128, 128, 1, 112, 112)),
    (512, 7168, 4096, False, ("pair", 256, 256, 1, 56, 112)),
    (8192, 8192, 8192, False, ("pair", 256, 256, 1, 1024, 148)),
    (1, 1024, 7168, False, ("split", 32, 64, 4, 16, 64)),
    (64, 960, 7168, False, ("split", 64, 64, 4, 15, 120)),
    (128, 2048, 7168, False, ("split", 128, 64, 2, 32, 128)),
    (1999, 2576, 1024, True, ("tile", 128, 128, 1, 336, 148)),
    (64, 1024, 7168, True, ("split", 64, 64, 4, 16, 64)),
    (40, 4096, 1040, False, ("split", 64, 64, 4, 64, 128)),  # K % 128 != 0
    (8, 1024, 4112, False, ("split", 32, 64, 4, 16, 64)),
    (40, 4096, 112, False, ("tile", 64, 64, 1, 64, 64))])
def test_plan(rrf, m, n, k, mx, want):
    p = rrf.rrf_plan_scaled_mm_act(m, n, k, 148, mx=mx)
    assert (p["kernel"], p["a_rows"], p["tile_n"], p["k_tiles_per_stage"], p["tiles"],
            p["ctas"]) == want


@pytest.mark.parametrize("sms", [148, 132, 40])
def test_plan_invariants(rrf, sms):
    for m in (1, 8, 9, 31, 33, 64, 65, 129, 300, 1000, 4096):
        for n in (16, 256, 1024, 4096, 7168, 16384):
            for k in (16, 128, 512, 1040, 2048, 7168):
                for mx in (False, True):
                    if mx and k % 128:
                        continue
                    p = rrf.rrf_plan_scaled_mm_act(m, n, k, sms, mx=mx)
                    kernel, rows, columns = p["kernel"], p["a_rows"], p["tile_n"]
                    high = 256 if kernel == "pair" else 128
                    if kernel != "swap":
                        assert p["tiles"] == -(-m // high) * -(-n // columns)
                    if kernel == "split":
                        split, left = divmod(p["ctas"], p["tiles"])
                        assert split in (2, 4, 8) and left == 0 and p["ctas"] <= sms
                        # every CTA has a part of K
                        z = p["k_tiles_per_stage"]
                        assert k >= 128 and -(-(k // 128) // z) + (k % 128 != 0) >= split
                        assert rows >= min(m, 128)
                    else:
                        assert p["ctas"] == min(p["tiles"], sms // 2) * 2 if kernel == "pair" \
                            else p["ctas"] == min(p["tiles"], sms)
                    if kernel == "tile":
                        assert (rows == 64) == (m <= 64 and not (columns == 128 and k < 128))


def test_plan_refusals(rrf):
    with pytest.raises(rrf.RrfError):
        rrf.rrf_plan_scaled_mm_act(8, 256, 1040, 148, mx=True)
    with pytest.raises(rrf.RrfError):
        rrf.rrf_plan_scaled_mm_act(8, 256, 1024, 1)
    assert rrf.rrf_plan_scaled_mm_act(0, 256, 1024, 148)["kernel"] is None


def test_erfc_polynomial():
    """The coefficients in the source: within 1.9e-6 of erfcx as they are
    written, and rounded to fp32 within 2^-24 of each term more; and the best
    fit: the error reaches its maximum eight times with alternating sign, which
    no polynomial of degree 6 betters."""
    import os
    import re

    import numpy as np
    import torch
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    text = open(os.path.join(root, "reduce_rmsnorm_fp8_b200", "csrc", "rrf_gemm.cu")).read()
    body = text[text.index("RRF_ACT_GELU) {"):]
    c = [float(x) for x in
         re.findall(r"both\((-?\d\.\d+e[+-]\d+)f\)", body[:body.index("const float2 e =")])]
    assert len(c) == 7  # from the highest power down
    a = np.linspace(0.0, 14.0, 140001)
    exact = torch.special.erfcx(torch.from_numpy(a) / np.sqrt(2.0)).numpy() / 2
    t = 1 / (1 + 0.3 * a)
    error = np.polyval(c, t) / exact - 1
    worst = np.abs(error).max()
    assert worst <= 1.9e-6
    rounded = np.polyval(np.float32(c).astype(np.float64), t) / exact - 1
    assert (np.abs(rounded) <= 1.9e-6 + 2.0 ** -24 * np.polyval(np.abs(c), t) / exact).all()
    runs = np.split(error, np.flatnonzero(np.diff(np.sign(error))) + 1)
    assert len(runs) == 8 and all(np.abs(r).max() >= 0.985 * worst for r in runs)


def test_the_library_builds_without_torch(rrf):
    """The C library does not need torch; only its Python binding does."""
    import os
    import subprocess
    import sys
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    code = ("import sys; sys.modules['torch'] = None\n"
            "from reduce_rmsnorm_fp8_b200 import build, lib\n"
            "assert build.build() == build.LIB and build.build_binding() is None\n"
            "print(lib.rrf_version().decode())")
    p = subprocess.run([sys.executable, "-c", code], cwd=root, capture_output=True, text=True,
                       timeout=600)
    assert p.returncode == 0 and p.stdout.strip() == "0.1.0", p.stdout + p.stderr
