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


def test_plan(rrf):
    """The plan follows the measured time of a round, for every shape: no other
    kernel's rounds would take less, and the CTAs cover the tiles."""
    cost = {("tile", 64, 64): (0.3, 0.24), ("tile", 128, 64): (0.7, 0.254),
            ("tile", 64, 128): (1.5, 0.26), ("tile", 128, 128): (2.0, 0.2875),
            ("pair", 256, 256): (5.0, 0.29)}
    seen = set()
    for m in (1, 8, 31, 33, 64, 65, 129, 300, 1000, 4096):
        for n in (16, 256, 1024, 7168, 16384):
            for k in (128, 1024, 7168):
                for mx in (False, True):
                    p = rrf.rrf_plan_scaled_mm_act(m, n, k, 148, mx=mx)
                    if m <= 32:
                        assert p == rrf.rrf_plan_scaled_mm(m, n, k, 148, mx=mx)
                        continue
                    key = (p["kernel"], p["a_rows"], p["tile_n"])
                    seen.add(key)
                    taken = {}
                    for (kernel, rows, columns), (e, c) in cost.items():
                        fits = m <= 64 if rows == 64 else m > 64 if rows == 128 else m > 128
                        if not fits:
                            continue
                        units, high = (74, 256) if kernel == "pair" else (148, 128)
                        tiles = -(-m // high) * -(-n // columns)
                        taken[kernel, rows, columns] = -(-tiles // units) * (e + k / 128 * c)
                        if (kernel, rows, columns) == key:
                            assert p["tiles"] == tiles
                            assert p["ctas"] == min(tiles, units) * (2 if kernel == "pair" else 1)
                    assert taken[key] <= min(taken.values()) + 1e-9
    assert seen == set(cost)
    # K % 128 != 0: one k-tile per box
    for m in (40, 100):
        assert rrf.rrf_plan_scaled_mm_act(m, 4096, 1040, 148)["k_tiles_per_stage"] == 1
    with pytest.raises(rrf.RrfError):
        rrf.rrf_plan_scaled_mm_act(8, 256, 1040, 148, mx=True)
