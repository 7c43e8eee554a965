"""Host validation of the per-head and cache calls, on made-up addresses: no
GPU is touched."""
import ctypes

import pytest


@pytest.fixture(scope="module")
def rrf():
    from reduce_rmsnorm_fp8_b200 import build
    build.build()
    import reduce_rmsnorm_fp8_b200 as m
    return m


MB = 1 << 20
T, HQ, HK, D, ROT = 10, 4, 2, 64, 32


def norm_case(**change):
    c = dict(q=MB, q_token=HQ * D, q_head=D, k=2 * MB, k_token=HK * D, k_head=D, q_out=3 * MB,
             q_out_token=HQ * D, q_out_head=D, k_out=4 * MB, k_out_token=HK * D, k_out_head=D,
             q_gamma=5 * MB, k_gamma=6 * MB, eps=1e-6, weight_offset=0.0, cos_sin=7 * MB,
             max_positions=100, rot_dim=ROT, positions=8 * MB, tokens=T, q_heads=HQ, kv_heads=HK,
             head_dim=D)
    assert set(change) <= set(c)
    return {**c, **change}


def packed(**change):
    """q, k and (elsewhere) v side by side in a token's row."""
    row = (HQ + 2 * HK) * D
    return norm_case(**{**dict(q_token=row, k_token=row, k=MB + HQ * D * 2), **change})


def cache_struct(rrf, pages=4, page=16, heads=HK, dim=D, codes=None, scales=None, **change):
    c = dict(k_codes=20 * MB, k_scales=21 * MB, v_codes=22 * MB, v_scales=23 * MB,
             num_pages=pages, page_size=page,
             code_strides=codes or (page * heads * dim, heads * dim, dim),
             scale_strides=scales or (page * heads, heads, 1))
    c.update(change)
    return bytes(rrf.RrfKvCache(*[tuple(v) if isinstance(v, (tuple, list)) else v
                                  for v in c.values()]))


def status(rrf, n):
    return rrf.Status(n).name


def check_norm(rrf, c):
    return status(rrf, rrf.lib.rrf_check_qk_norm_rope_args(*c.values()))


IN_PLACE = dict(q_out=MB, q_out_token=(HQ + 2 * HK) * D, k_out=MB + HQ * D * 2,
                k_out_token=(HQ + 2 * HK) * D)

NORM = [
    ({}, "OK"), (dict(tokens=0, q=None, cos_sin=None, q_out=None), "OK"),
    (dict(rot_dim=0, cos_sin=None, positions=None, max_positions=0), "OK"),
    (dict(q=None), "ERR_NULL"), (dict(k_out=None), "ERR_NULL"), (dict(k_gamma=None), "ERR_NULL"),
    (dict(cos_sin=None), "ERR_NULL"), (dict(positions=None), "ERR_NULL"),
    (dict(tokens=-1), "ERR_SHAPE"), (dict(tokens=2 ** 31), "ERR_SHAPE"),
    (dict(q_heads=0), "ERR_SHAPE"), (dict(kv_heads=0), "ERR_SHAPE"),
    (dict(q_heads=4097), "ERR_SHAPE"), (dict(head_dim=72), "ERR_SHAPE"),
    (dict(head_dim=528), "ERR_SHAPE"), (dict(head_dim=0), "ERR_SHAPE"),
    (dict(rot_dim=24), "ERR_SHAPE"), (dict(rot_dim=80), "ERR_SHAPE"),
    (dict(rot_dim=-16), "ERR_SHAPE"), (dict(max_positions=0), "ERR_SHAPE"),
    (dict(q_token=-256), "ERR_SHAPE"), (dict(q_head=1 << 41), "ERR_SHAPE"),
    (dict(eps=-1.0), "ERR_VALUE"), (dict(eps=float("nan")), "ERR_VALUE"),
    (dict(weight_offset=float("inf")), "ERR_VALUE"),
    (dict(q=MB + 8), "ERR_ALIGN"), (dict(k_token=HK * D + 4), "ERR_ALIGN"),
    (dict(q_out_head=D + 2), "ERR_ALIGN"), (dict(q_gamma=5 * MB + 2), "ERR_ALIGN"),
    (dict(cos_sin=7 * MB + 4), "ERR_ALIGN"), (dict(positions=8 * MB + 4), "ERR_ALIGN"),
    # an output's own heads on one another; the same is allowed of an input
    (dict(q_out_head=D - 8), "ERR_ALIAS"), (dict(k_out_token=0), "ERR_ALIAS"),
    (dict(q_token=0), "OK"), (dict(q_head=0), "OK"),
    # heads outermost
    (dict(q_out_token=D, q_out_head=T * D), "OK"),
    # outputs on inputs and on one another
    (dict(q_out=MB + 16), "ERR_ALIAS"), (dict(q_out=2 * MB), "ERR_ALIAS"),
    (dict(k_out=3 * MB), "ERR_ALIAS"), (dict(q_out=5 * MB), "ERR_ALIAS"),
    (dict(k_out=7 * MB), "ERR_ALIAS"), (dict(k_out=8 * MB), "ERR_ALIAS"),
    (dict(q_out=MB), "OK"), (dict(k_out=2 * MB), "OK"),
    (dict(q_out=MB, q_out_token=HQ * D + 8), "ERR_ALIAS"),
]


@pytest.mark.parametrize("change,want", NORM, ids=str)
def test_norm_rope_arguments(rrf, change, want):
    assert check_norm(rrf, norm_case(**change)) == want


@pytest.mark.parametrize("change,want", [
    ({}, "OK"), (IN_PLACE, "OK"),
    # queries in place, keys onto the values' part of the row, and onto the queries'
    ({**IN_PLACE, "k_out": MB + (HQ + HK) * D * 2}, "OK"),
    ({**IN_PLACE, "k_out": MB + (HQ - 1) * D * 2}, "ERR_ALIAS"),
    # the queries' output reaches into the keys' part of the next row
    (dict(q_out=MB + HQ * D * 2 + 16, q_out_token=(HQ + 2 * HK) * D), "ERR_ALIAS"),
], ids=str)
def test_parts_of_one_row(rrf, change, want):
    assert check_norm(rrf, packed(**change)) == want


def check_write(rrf, change=None, **cache):
    c = dict(k=MB, k_token=HK * D, k_head=D, v=2 * MB, v_token=HK * D, v_head=D, slots=8 * MB,
             scale_ub=1200.0, cache=cache_struct(rrf, **cache), tokens=T, kv_heads=HK, head_dim=D)
    c.update(change or {})
    return status(rrf, rrf.lib.rrf_check_kv_cache_write_args(*c.values()))


def test_cache_write_arguments(rrf):
    inf = float("inf")
    assert check_write(rrf) == "OK" and check_write(rrf, dict(scale_ub=inf)) == "OK"
    assert check_write(rrf, dict(tokens=0, k=None, cache=None)) == "OK"
    for change in (dict(k=None), dict(v=None), dict(slots=None), dict(cache=None)):
        assert check_write(rrf, change) == "ERR_NULL", change
    for name in ("k_codes", "k_scales", "v_codes", "v_scales"):
        assert check_write(rrf, **{name: None}) == "ERR_NULL", name
    for ub in (0.0, -1.0, float("nan")):
        assert check_write(rrf, dict(scale_ub=ub)) == "ERR_VALUE"
    for change in (dict(num_pages=0), dict(page_size=0), dict(num_pages=1 << 31),
                   dict(code_strides=(-16, HK * D, D)), dict(scale_strides=(1 << 41, HK, 1))):
        assert check_write(rrf, **change) == "ERR_SHAPE", change
    for change in (dict(k_codes=20 * MB + 8), dict(v_scales=23 * MB + 2),
                   dict(codes=(16 * HK * D, HK * D, D + 8))):
        assert check_write(rrf, **change) == "ERR_ALIGN", change
    assert check_write(rrf, dict(slots=8 * MB + 4)) == "ERR_ALIGN"
    # codes or scales on one another, on the other's, on an input
    for change in (dict(codes=(16 * HK * D, HK * D, 0)), dict(codes=(0, HK * D, D)),
                   dict(scales=(16 * HK, 0, 1)), dict(v_codes=20 * MB + 64),
                   dict(v_scales=21 * MB), dict(k_scales=20 * MB), dict(v_codes=MB),
                   dict(k_scales=8 * MB)):
        assert check_write(rrf, **change) == "ERR_ALIAS", change


def test_cache_layouts(rrf):
    """Head-major pages, keys and values in one buffer by page, a part of a
    wider cache."""
    assert check_write(rrf, codes=(HK * 16 * D, D, 16 * D), scales=(HK * 16, 1, 16)) == "OK"
    page = HK * 16 * D
    both = dict(codes=(2 * page, HK * D, D), v_codes=20 * MB + page)
    assert check_write(rrf, **both) == "OK"
    assert check_write(rrf, **{**both, "v_codes": 20 * MB + page - 16}) == "ERR_ALIAS"
    assert check_write(rrf, codes=(16 * 5 * D, 5 * D, D)) == "OK"


def test_fused_arguments(rrf):
    def check(change=None, **cache):
        n = norm_case(**{k: v for k, v in (change or {}).items() if k in norm_case()})
        extra = {k: v for k, v in (change or {}).items() if k not in n}
        e = dict(v=9 * MB, v_token=HK * D, v_head=D, slots=10 * MB, scale_ub=1200.0,
                 cache=cache_struct(rrf, **cache))
        e.update(extra)
        v = list(n.values())
        return status(rrf, rrf.lib.rrf_check_qk_norm_rope_kv_cache_args(
            *v[:6], e["v"], e["v_token"], e["v_head"], *v[6:9], *v[12:20], e["slots"],
            e["scale_ub"], e["cache"], *v[20:]))

    assert check() == "OK" and check(dict(q_out=MB)) == "OK"
    assert check(dict(tokens=0, v=None, cache=None)) == "OK"
    for change, want in [(dict(v=None), "ERR_NULL"), (dict(slots=None), "ERR_NULL"),
                         (dict(cache=None), "ERR_NULL"), (dict(positions=None), "ERR_NULL"),
                         (dict(scale_ub=0.0), "ERR_VALUE"), (dict(eps=-1.0), "ERR_VALUE"),
                         (dict(rot_dim=8), "ERR_SHAPE"), (dict(kv_heads=0), "ERR_SHAPE"),
                         (dict(v=9 * MB + 2), "ERR_ALIGN"), (dict(q_out=9 * MB), "ERR_ALIAS"),
                         (dict(q_out=2 * MB), "ERR_ALIAS"), (dict(q_out=20 * MB), "ERR_ALIAS"),
                         (dict(q_out=10 * MB), "ERR_ALIAS")]:
        assert check(change) == want, change
    assert check(None, k_codes=2 * MB) == "ERR_ALIAS"
    assert check(None, v_scales=7 * MB) == "ERR_ALIAS"


def test_cache_read_arguments(rrf):
    def check(change=None, **cache):
        c = dict(cache=cache_struct(rrf, **cache), block_table=MB, table_stride=5, table_width=5,
                 seq_starts=2 * MB, sequences=3, k_out=3 * MB, v_out=4 * MB, rows=50,
                 kv_heads=HK, head_dim=D)
        c.update(change or {})
        return status(rrf, rrf.lib.rrf_check_kv_cache_read_args(*c.values()))

    assert check() == "OK"
    assert check(dict(rows=0, k_out=None)) == "OK" and check(dict(sequences=0)) == "OK"
    assert check(dict(table_width=0, block_table=None)) == "OK"
    for change, want in [(dict(block_table=None), "ERR_NULL"), (dict(seq_starts=None), "ERR_NULL"),
                         (dict(v_out=None), "ERR_NULL"), (dict(cache=None), "ERR_NULL"),
                         (dict(rows=-1), "ERR_SHAPE"), (dict(sequences=-1), "ERR_SHAPE"),
                         (dict(table_width=-1), "ERR_SHAPE"), (dict(table_stride=-5), "ERR_SHAPE"),
                         (dict(head_dim=40), "ERR_SHAPE"), (dict(k_out=3 * MB + 8), "ERR_ALIGN"),
                         (dict(block_table=MB + 2), "ERR_ALIGN"),
                         (dict(seq_starts=2 * MB + 1), "ERR_ALIGN"),
                         (dict(v_out=3 * MB), "ERR_ALIAS"), (dict(k_out=20 * MB), "ERR_ALIAS"),
                         (dict(k_out=MB), "ERR_ALIAS"), (dict(v_out=2 * MB), "ERR_ALIAS"),
                         (dict(v_out=23 * MB), "ERR_ALIAS")]:
        assert check(change) == want, change
    # a cache that is only read may lie on itself (a broadcast page)
    assert check(None, codes=(0, HK * D, D)) == "OK"


def test_cpu_tensors_are_refused(rrf):
    import torch
    q = torch.zeros((2, 2, 64), dtype=torch.bfloat16)
    gamma = torch.zeros(64, dtype=torch.bfloat16)
    with pytest.raises(ValueError):
        rrf.rrf_qk_norm_rope(q, q, gamma, gamma, 1e-6, 0.0, None, None)
    slots = torch.zeros(2, dtype=torch.int64)
    codes = torch.zeros((1, 16, 2, 64), dtype=torch.uint8).view(torch.float8_e4m3fn)
    scales = torch.zeros((1, 16, 2))
    with pytest.raises(ValueError):
        rrf.rrf_kv_cache_write_fp8(q, q, slots, codes, scales, codes, scales)
    with pytest.raises(ValueError):
        rrf.rrf_kv_cache_read_fp8(codes, scales, codes, scales, slots.int()[None],
                                  slots.int(), q, q)


def test_rope_table():
    import math

    import torch
    from reduce_rmsnorm_fp8_b200 import rope_table
    t = rope_table(50, 32, theta=1000.0, device="cpu")
    assert t.shape == (50, 32) and t.dtype == torch.float32
    for p in (0, 1, 49):
        for i in (0, 7, 15):
            a = p * 1000.0 ** (-2.0 * i / 32)
            assert abs(float(t[p, i]) - math.cos(a)) <= 2.0 ** -24
            assert abs(float(t[p, 16 + i]) - math.sin(a)) <= 2.0 ** -24
    with pytest.raises(ValueError):
        rope_table(5, 24, device="cpu")


def test_constants_match_the_header(rrf):
    import os
    import re
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    text = open(os.path.join(root, "include", "rrf.h")).read()
    for name in ("RRF_DEVICE_ERROR_INDEX", "RRF_MAX_HEAD_DIM"):
        assert getattr(rrf, name) == int(re.search(rf"#define {name} (\d+)u?", text).group(1))
    assert ctypes.sizeof(rrf.RrfKvCache) == 4 * 8 + 2 * 8 + 6 * 8


def test_tensors_that_require_grad_are_refused(rrf):
    """Where autograd records, before anything else of the tensor is looked at;
    under no_grad the next check speaks (these are CPU tensors)."""
    import torch
    x = torch.zeros((2, 2, 64), dtype=torch.bfloat16)
    w = torch.zeros((2, 2, 64), dtype=torch.bfloat16, requires_grad=True)
    gamma = torch.zeros(64, dtype=torch.bfloat16)
    slots = torch.zeros(2, dtype=torch.int64)
    codes = torch.zeros((1, 16, 2, 64), dtype=torch.uint8).view(torch.float8_e4m3fn)
    scales = torch.zeros((1, 16, 2))
    a, row = torch.zeros((2, 128)).to(torch.float8_e4m3fn), torch.ones(2)
    square = torch.zeros((2, 2), dtype=torch.bfloat16, requires_grad=True)
    for call, name in (
            (lambda: rrf.rrf_qk_norm_rope(w, x, gamma, gamma, 1e-6, 0.0, None, None), "q"),
            (lambda: rrf.rrf_qk_norm_rope(x, w, gamma, gamma, 1e-6, 0.0, None, None), "k"),
            (lambda: rrf.rrf_kv_cache_write_fp8(x, w, slots, codes, scales, codes, scales), "v"),
            (lambda: rrf.rrf_qk_norm_rope_kv_cache_fp8(x, x, w, gamma, gamma, 1e-6, 0.0, None,
                                                       None, slots, codes, scales, codes,
                                                       scales), "v"),
            (lambda: rrf.rrf_scaled_mm_fp8_act(a, row.clone().requires_grad_(), a, row),
             "a_scale"),
            (lambda: rrf.rrf_scaled_mm_fp8_act(a, row, a, row, bias=square[0]), "bias"),
            (lambda: rrf.rrf_scaled_mm_fp8_act(a, row, a, row, residual=square), "residual"),
            (lambda: rrf.rrf_scaled_mm_mxfp8_act(a, row, a, row, out=square), "out"),
            (lambda: rrf.rrf_kv_cache_read_fp8(codes, scales, codes, scales, slots.int()[None],
                                               slots.int(), w, x), "k_out")):
        with pytest.raises(ValueError, match=f"^{name} must be .*require grad"):
            call()
        with torch.no_grad(), pytest.raises(ValueError, match="CUDA tensor"):
            call()
