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
