"""GPU parity of the per-head norm with rotation and of the FP8 key / value
cache against float64 (tests/heads_reference.py derives the tolerances)."""
import pytest
import torch

import heads_reference as ref

pytestmark = pytest.mark.gpu
INF = float("inf")


@pytest.fixture(scope="module")
def rrf():
    import reduce_rmsnorm_fp8_b200 as m
    m.rrf_device_error(clear=True)
    yield m
    assert m.rrf_device_error() == 0


def gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def randn(g, *shape):
    return torch.randn(shape, generator=g, device="cuda")


def problem(seed, tokens, hq, hk, dim, rot, wo=0.0, positions=1000):
    """Parts of a packed projection, gammas, table, positions."""
    from reduce_rmsnorm_fp8_b200 import rope_table
    g = gen(seed)
    qkv = randn(g, tokens, hq + 2 * hk, dim).mul_(1.7).bfloat16()
    gammas = [(0.2 * randn(g, dim) + 1 - wo).bfloat16() for _ in range(2)]
    table = rope_table(positions, rot) if rot else None
    pos = torch.randint(positions, (tokens,), generator=g, device="cuda")
    return qkv[:, :hq], qkv[:, hq:hq + hk], qkv[:, hq + hk:], *gammas, table, pos


def cpu(t):
    return None if t is None else t.detach().cpu()


def check_norm(got, x, gamma, eps, wo, table, pos, interleaved, label):
    y, mag = ref.norm_rope(cpu(x), cpu(gamma), eps, wo, cpu(table), cpu(pos), interleaved)
    ref.check_bf16(cpu(got), y, ref.norm_error(mag), label)


def new_cache(g, pages, page, heads, dim, layout="nhd"):
    out = []
    for _ in range(2):
        codes = randn(g, pages, page, heads, dim).to(torch.float8_e4m3fn)
        if layout == "hnd":
            codes = codes.view(pages, heads, page, dim).transpose(1, 2)
        elif layout == "gaps":  # a part of a wider cache
            wide = torch.zeros((pages, page, 2 * heads + 1, dim), dtype=torch.uint8,
                               device="cuda").view(torch.float8_e4m3fn)
            wide.view(torch.uint8)[:, :, 1:heads + 1] = codes.view(torch.uint8)
            codes = wide[:, :, 1:heads + 1]
        scales = torch.rand((pages, page, heads), generator=g, device="cuda")
        if layout == "hnd":
            scales = scales.view(pages, heads, page).transpose(1, 2)
        out += [codes, scales]
    return out


def clone_cache(cache):
    return [t.view(torch.uint8 if t.dtype == torch.float8_e4m3fn else t.dtype).clone()
            for t in cache]


def draw_slots(g, tokens, total, padding):
    slots = torch.randperm(total, generator=g, device="cuda")[:tokens]
    drop = torch.rand(tokens, generator=g, device="cuda") < padding
    return torch.where(drop, -1 - slots, slots)


def check_cache(cache, before, slots, k, kerr, v, scale_ub, exact_v=True, label=""):
    """The named slots hold k and v (float64, CPU); every other byte is as
    before."""
    page_size = cache[0].shape[1]
    slots = cpu(slots)
    keep = slots >= 0
    page, place = ref.place_of(slots[keep], page_size)
    for n, (x, err) in enumerate(((k, kerr), (v, torch.zeros_like(v)))):
        codes, scales = cpu(cache[2 * n]), cpu(cache[2 * n + 1])
        values = codes.view(torch.uint8)[page, place].view(torch.float8_e4m3fn).double()
        ref.check_codes(values, scales[page, place], x[keep], err[keep], scale_ub,
                        f"{label} {'kv'[n]}")
        if n == 1 and exact_v:
            assert torch.equal(values, ref.exact_codes(x[keep], scale_ub)), \
                f"{label}: a code is not the nearest"
        rest = torch.ones(codes.shape[:2], dtype=torch.bool)
        rest[page, place] = False
        assert torch.equal(codes.view(torch.uint8)[rest], cpu(before[2 * n])[rest]), label
        assert torch.equal(scales[rest], cpu(before[2 * n + 1])[rest]), label


SHAPES = [  # tokens, q heads, kv heads, dim, rot
    (1, 8, 1, 128, 128), (2, 1, 1, 16, 16), (37, 12, 3, 80, 32), (5, 7, 7, 64, 64),
    (300, 8, 2, 128, 64), (3, 5, 1, 96, 96), (19, 3, 2, 192, 64), (33, 4, 4, 256, 256),
    (7, 2, 1, 272, 16), (4, 3, 3, 512, 512), (65, 9, 5, 48, 48), (11, 33, 17, 32, 16),
    (6, 4, 2, 128, 0), (1000, 1, 1, 64, 32), (23, 13, 7, 160, 96), (9, 11, 11, 144, 144),
    (50, 21, 1, 48, 16), (4, 6, 6, 112, 112)]


@pytest.mark.parametrize("shape", SHAPES, ids=str)
@pytest.mark.parametrize("interleaved", [False, True])
def test_norm_rope(rrf, shape, interleaved):
    tokens, hq, hk, dim, rot = shape
    wo = 1.0 if dim % 3 == 0 else 0.0
    q, k, _, qg, kg, table, pos = problem(dim + tokens, tokens, hq, hk, dim, rot, wo)
    qo, ko = rrf.rrf_qk_norm_rope(q, k, qg, kg, 1e-5, wo, table, pos, interleaved=interleaved)
    check_norm(qo, q, qg, 1e-5, wo, table, pos, interleaved, "q")
    check_norm(ko, k, kg, 1e-5, wo, table, pos, interleaved, "k")


@pytest.mark.parametrize("shape", SHAPES, ids=str)
@pytest.mark.parametrize("page,layout", [(16, "nhd"), (7, "hnd"), (1, "nhd"), (5, "gaps")])
def test_cache_write(rrf, shape, page, layout):
    tokens, _, hk, dim, _ = shape
    g = gen(tokens * 7 + dim)
    kv = randn(g, tokens, 2 * hk, dim).bfloat16()
    k, v = kv[:, :hk], kv[:, hk:]
    pages = 2 + 2 * tokens // page
    cache = new_cache(g, pages, page, hk, dim, layout)
    slots = draw_slots(g, tokens, pages * page, 0.2)
    before = clone_cache(cache)
    rrf.rrf_kv_cache_write_fp8(k, v, slots, *cache)
    kd, vd = cpu(k).double(), cpu(v).double()
    check_cache(cache, before, slots, kd, torch.zeros_like(kd), vd, INF, label=layout)


@pytest.mark.parametrize("shape", SHAPES, ids=str)
@pytest.mark.parametrize("interleaved,layout", [(False, "nhd"), (True, "hnd")])
def test_fused(rrf, shape, interleaved, layout):
    tokens, hq, hk, dim, rot = shape
    q, k, v, qg, kg, table, pos = problem(3 * dim + tokens, tokens, hq, hk, dim, rot)
    g = gen(5)
    cache = new_cache(g, 3 + tokens // 4, 16, hk, dim, layout)
    slots = draw_slots(g, tokens, (3 + tokens // 4) * 16, 0.2)
    before = clone_cache(cache)
    qo = rrf.rrf_qk_norm_rope_kv_cache_fp8(q, k, v, qg, kg, 1e-6, 0.0, table, pos, slots, *cache,
                                           scale_ub=2.5, interleaved=interleaved)
    check_norm(qo, q, qg, 1e-6, 0.0, table, pos, interleaved, "q")
    y, mag = ref.norm_rope(cpu(k), cpu(kg), 1e-6, 0.0, cpu(table), cpu(pos), interleaved)
    check_cache(cache, before, slots, y, ref.norm_error(mag), cpu(v).double(), 2.5,
                exact_v=False, label=layout)


def test_fused_is_the_two_calls(rrf):
    """Queries bit for bit; values bit for bit; keys differ from the two-call
    form only by its rounding to bf16 between."""
    q, k, v, qg, kg, table, pos = problem(8, 129, 6, 2, 128, 128)
    g = gen(9)
    one, two = new_cache(g, 20, 16, 2, 128), new_cache(g, 20, 16, 2, 128)
    slots = draw_slots(g, 129, 320, 0.0)
    qo = rrf.rrf_qk_norm_rope_kv_cache_fp8(q, k, v, qg, kg, 1e-6, 0.0, table, pos, slots, *one)
    q2, k2 = rrf.rrf_qk_norm_rope(q, k, qg, kg, 1e-6, 0.0, table, pos)
    rrf.rrf_kv_cache_write_fp8(k2, v, slots, *two)
    assert torch.equal(qo, q2)
    at = ref.place_of(slots, 16)
    assert torch.equal(one[2].view(torch.uint8)[at], two[2].view(torch.uint8)[at])
    assert torch.equal(one[3][at], two[3][at])
    # the maximum was rounded to bf16 between, and in the one pass was not
    assert bool(((one[1][at] - two[1][at]).abs() <= 1.01 * ref.H * one[1][at]).all())


def test_in_place_and_head_major(rrf):
    q, k, v, qg, kg, table, pos = problem(10, 70, 5, 3, 96, 96)
    want = rrf.rrf_qk_norm_rope(q, k, qg, kg, 1e-6, 0.0, table, pos)
    # heads outermost, in and out
    qt, kt = (x.transpose(0, 1).contiguous().transpose(0, 1) for x in (q, k))
    out = torch.zeros((5, 70, 96), dtype=torch.bfloat16, device="cuda")
    got = rrf.rrf_qk_norm_rope(qt, kt, qg, kg, 1e-6, 0.0, table, pos, q_out=out.transpose(0, 1))
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    keep = v.clone()
    got = rrf.rrf_qk_norm_rope(q, k, qg, kg, 1e-6, 0.0, table, pos, q_out=q, k_out=k)
    assert got[0] is q and torch.equal(q, want[0]) and torch.equal(k, want[1])
    assert torch.equal(v, keep)


def test_far_positions(rrf):
    """The table holds the angles of far positions to fp32."""
    n = 1 << 18
    q, k, _, qg, kg, _, _ = problem(11, 9, 2, 1, 64, 0)
    table = rrf.rope_table(n, 64, theta=5e5)
    pos = torch.tensor([0, 1, n - 1, n - 2, n // 2, 3, 99999, 100000, 7], device="cuda")
    qo, _ = rrf.rrf_qk_norm_rope(q, k, qg, kg, 1e-6, 0.0, table, pos)
    angle = cpu(pos).double()[:, None] * torch.pow(
        torch.tensor(5e5, dtype=torch.float64), -torch.arange(32, dtype=torch.float64) / 32)
    exact = torch.cat((angle.cos(), angle.sin()), 1)
    # one rounding to fp32, and the last place of the two libraries' angles
    assert float((cpu(table)[cpu(pos)].double() - exact).abs().max()) <= U2
    y, mag = ref.norm_rope(cpu(q), cpu(qg), 1e-6, 0.0, exact, torch.arange(9), False)
    ref.check_bf16(cpu(qo), y, ref.norm_error(mag) + U2 * 2 * mag.amax(-1, keepdim=True), "far")


# 2^-24 of a value up to 1, and angles up to 2^18 off by a few steps of float64
U2 = 2.0 ** -24 + 2.0 ** 18 * 2.0 ** -50


SPECIAL = {
    "zero": lambda d: torch.zeros(d),
    "minus zero": lambda d: -torch.zeros(d),
    "tiny": lambda d: torch.full((d,), 1e-38),
    "below the floor": lambda d: torch.linspace(-9e-13, 9e-13, d),
    "largest": lambda d: torch.where(torch.arange(d) % 3 == 0, -3.3e38, 1e37),
    "one large": lambda d: torch.where(torch.arange(d) == d - 1, 3e38, 1.0),
    "over 1e30": lambda d: torch.linspace(-1e31, 1e31, d),
    "nan": lambda d: torch.where(torch.arange(d) == 3, float("nan"), 1.5),
    "all nan": lambda d: torch.full((d,), float("nan")),
    "infinite": lambda d: torch.where(torch.arange(d) == 5, -INF, 2.0),
}


@pytest.mark.parametrize("scale_ub", [INF, 1200.0, 0.01])
@pytest.mark.parametrize("dim", [64, 80])
def test_special_rows_of_the_cache(rrf, scale_ub, dim):
    x = torch.stack([f(dim) for f in SPECIAL.values()]).bfloat16()[:, None].cuda()
    n = x.shape[0]
    cache = new_cache(gen(1), n, 1, 1, dim)
    rrf.rrf_kv_cache_write_fp8(x, x, torch.arange(n, device="cuda"), *cache, scale_ub=scale_ub)
    xd = cpu(x)[:, 0].double()
    amax = torch.where(xd.isnan(), 0.0, xd.abs()).amax(-1).clamp(max=scale_ub).clamp(min=1e-12)
    for codes, scales in ((cache[0], cache[1]), (cache[2], cache[3])):
        s = cpu(scales)[:, 0, 0].double()
        v = cpu(codes)[:, 0, 0].double()
        for i, name in enumerate(SPECIAL):
            m = float(amax[i])
            if m == INF:  # finite values 0, infinities NaN
                assert float(s[i]) == INF and bool((v[i].isnan() == xd[i].isinf()).all()), name
                assert bool((v[i][~xd[i].isinf()] == 0).all()), name
                continue
            assert abs(float(s[i]) * 448 - m) <= 1.01 * ref.U * m, name
            assert torch.equal(v[i].isnan(), xd[i].isnan()), name
            y = (xd[i].clamp(-m, m) / (m / 448))
            ok = ~xd[i].isnan()
            step = torch.exp2(torch.floor(torch.log2(y.abs().clamp(min=2.0 ** -6))) - 3)
            assert bool(((v[i] - y).abs()[ok] <= (step / 2 + 4 * ref.U * y.abs())[ok]).all()), name


@pytest.mark.parametrize("scale_ub", [2.0 ** e for e in (28, 29, 30, 66, 100, 127)])
@pytest.mark.parametrize("dim", [64, 80])
def test_special_rows_under_a_large_bound(rrf, scale_ub, dim):
    """A finite bound cuts an infinity however large it is: 448 times it, as a
    quotient, may pass fp32.  (Powers of two: the bound itself is not rounded.)"""
    test_special_rows_of_the_cache(rrf, scale_ub, dim)
    # the values of the one pass go by the same rule
    x = torch.stack([f(dim) for f in SPECIAL.values()]).bfloat16()[:, None].cuda()
    n = x.shape[0]
    one, two = new_cache(gen(1), n, 1, 1, dim), new_cache(gen(1), n, 1, 1, dim)
    slots, gamma = torch.arange(n, device="cuda"), torch.ones(dim, device="cuda").bfloat16()
    y = torch.ones_like(x)
    rrf.rrf_kv_cache_write_fp8(y, x, slots, *one, scale_ub=scale_ub)
    rrf.rrf_qk_norm_rope_kv_cache_fp8(y, y, x, gamma, gamma, 0.0, 0.0, None, None, slots, *two,
                                      scale_ub=scale_ub)
    assert torch.equal(one[2].view(torch.uint8), two[2].view(torch.uint8))
    assert torch.equal(one[3], two[3])


def test_special_rows_of_the_norm(rrf):
    dim = 64
    q, k, _, qg, kg, table, pos = problem(12, 4, 2, 1, dim, 64)
    q = q.clone()
    q[0, 0] = 0
    q[1, 1] = float("nan")
    q[2, 0, 7] = INF
    qo, _ = rrf.rrf_qk_norm_rope(q, k, qg, kg, 1e-6, 0.0, table, pos)
    assert bool((qo[0, 0] == 0).all()) and bool(qo[1, 1].isnan().all())
    # sum of squares infinite: finite values 0, the infinity NaN, so its pair too
    bad = torch.zeros(dim, dtype=torch.bool)
    bad[[7, 39]] = True
    assert torch.equal(cpu(qo[2, 0]).isnan(), bad)
    assert bool((qo[2, 0][~bad.cuda()] == 0).all())
    # the other heads of those tokens are not touched by them
    check_norm(qo[3:], q[3:], qg, 1e-6, 0.0, table, pos[3:], False, "clean")
    check_norm(qo[:1, 1:], q[:1, 1:], qg, 1e-6, 0.0, table, pos[:1], False, "clean")


@pytest.mark.parametrize("bad", [-1, 1000, 1 << 40, -(1 << 62)])
def test_positions_outside_the_table_are_left_out(rrf, bad):
    q, k, v, qg, kg, table, pos = problem(13, 6, 2, 1, 64, 64)
    pos = pos.clone()
    pos[4] = bad
    qo, ko = torch.full_like(q, 7.0), torch.full_like(k, 7.0)
    rrf.rrf_qk_norm_rope(q, k, qg, kg, 1e-6, 0.0, table, pos, q_out=qo, k_out=ko)
    assert rrf.rrf_device_error(clear=True) == rrf.RRF_DEVICE_ERROR_INDEX
    assert bool((qo[4] == 7).all()) and bool((ko[4] == 7).all())
    ok = torch.tensor([0, 1, 2, 3, 5], device="cuda")
    check_norm(qo[ok], q[ok], qg, 1e-6, 0.0, table, pos[ok], False, "others")


def test_slots_outside_the_cache_are_left_out(rrf):
    g = gen(14)
    kv = randn(g, 6, 2, 64).bfloat16()
    cache = new_cache(g, 4, 16, 1, 64)
    before = clone_cache(cache)
    slots = torch.tensor([0, 64, 63, 1 << 40, -1, -(1 << 62)], device="cuda")
    rrf.rrf_kv_cache_write_fp8(kv[:, :1], kv[:, 1:], slots, *cache)
    assert rrf.rrf_device_error(clear=True) == rrf.RRF_DEVICE_ERROR_INDEX
    named = torch.where((slots >= 0) & (slots < 64), slots, -1)
    kd = cpu(kv).double()
    check_cache(cache, before, named, kd[:, :1], torch.zeros_like(kd[:, :1]), kd[:, 1:], INF)


# ------------------------------------------------------------------- read ---

def read_problem(seed, lens, pages, page, heads, dim, layout="nhd", spare=3, width=0):
    g = gen(seed)
    cache = new_cache(g, pages, page, heads, dim, layout)
    need = [-(-n // page) for n in lens]
    table = torch.full((len(lens), max(need + [width])), -7, dtype=torch.int32)
    for s, n in enumerate(need):
        # a page may be named by several sequences
        table[s, :n] = torch.randint(pages, (n,), generator=torch.Generator().manual_seed(s))
    starts = torch.tensor([0] + list(lens)).cumsum(0).int()
    rows = sum(lens) + spare
    out = [torch.full((rows, heads, dim), 3.0 + i, dtype=torch.bfloat16, device="cuda")
           for i in range(2)]
    return cache, table.cuda(), starts.cuda(), out


def check_read(cache, table, starts, out, first=0):
    table, starts = cpu(table), cpu(starts).long()
    page_size = cache[0].shape[1]
    covered = torch.zeros(out[0].shape[0], dtype=torch.bool)
    rows, pg, pl = [], [], []
    for s in range(len(starts) - 1):
        for t in range(int(starts[s + 1] - starts[s])):
            r = int(starts[s]) + t
            if r < len(covered):
                rows.append(r)
                pg.append(int(table[s, t // page_size]))
                pl.append(t % page_size)
    covered[rows] = True
    for n in range(2):
        codes = cpu(cache[2 * n]).view(torch.uint8)[pg, pl].view(torch.float8_e4m3fn).double()
        y = codes * cpu(cache[2 * n + 1])[pg, pl].double()[..., None]
        ref.check_bf16(cpu(out[n])[rows], y, ref.U * y.abs(), "kv"[n])
        assert bool((out[n][~covered.cuda()] == 3.0 + n).all()), "a row of no sequence changed"


@pytest.mark.parametrize("lens", [[1], [0], [0, 5, 0, 0, 17, 0], [16, 16], [33, 1, 70, 2],
                                  [3] * 300, [0] * 700 + [40] + [0] * 40, [2500, 1]], ids=str)
@pytest.mark.parametrize("page,heads,dim,layout", [(16, 2, 64, "nhd"), (7, 1, 16, "hnd"),
                                                   (1, 3, 80, "nhd"), (64, 8, 128, "gaps"),
                                                   (5, 5, 272, "nhd")])
def test_read(rrf, lens, page, heads, dim, layout):
    p = read_problem(len(lens), lens, 9, page, heads, dim, layout)
    got = rrf.rrf_kv_cache_read_fp8(*p[0], p[1], p[2], *p[3])
    assert got[0] is p[3][0]
    check_read(*p)


def test_read_of_fewer_rows_and_wide_tables(rrf):
    cache, table, starts, out = read_problem(1, [20, 30], 9, 16, 2, 64, width=40)
    out = [o[:41].clone() for o in out]  # the second sequence does not fit
    wide = torch.full((2, 90), -1, dtype=torch.int32, device="cuda")
    wide[:, 10:50] = table
    rrf.rrf_kv_cache_read_fp8(*cache, wide[:, 10:50], starts, *out)
    check_read(cache, table, starts, out)
    # rows before the first sequence belong to none
    out = [torch.full_like(o, 3.0 + i) for i, o in enumerate(out)]
    rrf.rrf_kv_cache_read_fp8(*cache, table, starts + 4, *out)
    check_read(cache, table, starts + 4, out)


@pytest.mark.parametrize("which", [0, 1])
def test_read_to_outputs_aligned_to_16_bytes(rrf, which):
    cache, table, starts, out = read_problem(3, [20, 5], 9, 16, 3, 80)
    n = out[which].numel()
    odd = torch.full((n + 16,), 3.0 + which, dtype=torch.bfloat16, device="cuda")
    at = 8 if odd.data_ptr() % 32 == 0 else 16
    out[which] = odd[at:at + n].view(out[which].shape)
    assert out[which].data_ptr() % 32 == 16
    rrf.rrf_kv_cache_read_fp8(*cache, table, starts, *out)
    check_read(cache, table, starts, out)
    assert bool((odd[:at] == 3 + which).all()) and bool((odd[at + n:] == 3 + which).all())


@pytest.mark.parametrize("bad", [-1, 9, 2 ** 31 - 1, -2 ** 31])
def test_pages_outside_the_cache_are_left_out(rrf, bad):
    cache, table, starts, out = read_problem(2, [20, 5], 9, 16, 2, 64)
    want = [o.clone() for o in out]
    rrf.rrf_kv_cache_read_fp8(*cache, table, starts, *want)
    table[0, 1] = bad
    rrf.rrf_kv_cache_read_fp8(*cache, table, starts, *out)
    assert rrf.rrf_device_error(clear=True) == rrf.RRF_DEVICE_ERROR_INDEX
    for n in range(2):
        assert bool((out[n][16:20] == 3.0 + n).all())
        assert torch.equal(out[n][:16], want[n][:16]) and torch.equal(out[n][20:], want[n][20:])
    # a table too narrow for its sequence
    rrf.rrf_kv_cache_read_fp8(*cache, table[:, :1], starts, *out)
    assert rrf.rrf_device_error(clear=True) == rrf.RRF_DEVICE_ERROR_INDEX
    assert bool((out[0][16:20] == 3.0).all())


def test_offsets_past_32_bits(rrf):
    """A cache of more than 2^32 codes for each of keys and values."""
    heads, dim, page = 8, 128, 16
    pages = 2 ** 32 // (heads * dim * page) + 3
    cache = []
    for _ in range(2):
        cache += [torch.zeros((pages, page, heads, dim), dtype=torch.uint8,
                              device="cuda").view(torch.float8_e4m3fn),
                  torch.zeros((pages, page, heads), device="cuda")]
    g = gen(3)
    kv = randn(g, 4, 2 * heads, dim).bfloat16()
    slots = torch.tensor([0, pages * page - 1, pages * page - 40, 2 ** 31 // (heads * dim)],
                         device="cuda")
    rrf.rrf_kv_cache_write_fp8(kv[:, :heads], kv[:, heads:], slots, *cache)
    page_of, place = ref.place_of(slots, page)
    for n in range(2):
        x = cpu(kv[:, n * heads:(n + 1) * heads]).double()
        codes = cpu(cache[2 * n].view(torch.uint8)[page_of, place]).view(torch.float8_e4m3fn)
        assert torch.equal(codes.double(), ref.exact_codes(x, INF))
        assert int((cache[2 * n + 1] != 0).sum()) == 4 * heads
    out = [torch.zeros((page, heads, dim), dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    table = torch.tensor([[pages - 1]], dtype=torch.int32, device="cuda")
    rrf.rrf_kv_cache_read_fp8(*cache, table, torch.tensor([0, page], device="cuda").int(), *out)
    y = cpu(cache[0][pages - 1, page - 1]).double() * cpu(cache[1][pages - 1, page - 1])[:, None]
    ref.check_bf16(cpu(out[0][-1]), y, ref.U * y.abs(), "far page")
    assert bool((out[0][:page - 1] == 0).all())


# ------------------------------------------------------ together, in streams ---

def step(rrf, s):
    """A layer's step: projection, heads into the cache, the batch read back."""
    qkv = rrf.rrf_scaled_mm_fp8(s["a"], s["a_scale"], s["b"], s["b_scale"], out=s["qkv"])
    qkv = qkv.view(-1, s["hq"] + 2 * s["hk"], s["dim"])
    q, k, v = qkv.split((s["hq"], s["hk"], s["hk"]), dim=1)
    rrf.rrf_qk_norm_rope_kv_cache_fp8(q, k, v, s["qg"], s["kg"], 1e-6, 0.0, s["table"], s["pos"],
                                      s["slots"], *s["cache"], q_out=s["q_out"])
    rrf.rrf_kv_cache_read_fp8(*s["cache"], s["block_table"], s["starts"], *s["out"])


def step_problem(rrf, seed, tokens=48, hq=4, hk=2, dim=64, hidden=512):
    import workloads
    m = workloads.make_gemm_case(tokens, (hq + 2 * hk) * dim, hidden, sub=seed, bias=False,
                                 device="cuda")
    g = gen(seed)
    bf16 = dict(dtype=torch.bfloat16, device="cuda")
    pages = tokens // 16
    order = torch.randperm(pages, generator=g, device="cuda")
    i = torch.arange(tokens, device="cuda")
    return dict(a=m.a, a_scale=m.a_scale, b=m.b, b_scale=m.b_scale, hq=hq, hk=hk, dim=dim,
                qkv=torch.empty((tokens, (hq + 2 * hk) * dim), **bf16),
                qg=(1 + 0.1 * randn(g, dim)).bfloat16(), kg=(1 + 0.1 * randn(g, dim)).bfloat16(),
                table=rrf.rope_table(tokens, dim), pos=i, slots=order[i // 16] * 16 + i % 16,
                cache=new_cache(g, pages, 16, hk, dim), block_table=order.int()[None],
                starts=torch.tensor([0, tokens], dtype=torch.int32, device="cuda"),
                q_out=torch.empty((tokens, hq, dim), **bf16),
                out=[torch.empty((tokens, hk, dim), **bf16) for _ in range(2)])


def check_step(s):
    qkv = s["qkv"].view(-1, s["hq"] + 2 * s["hk"], s["dim"])
    q, k, v = (cpu(x) for x in qkv.split((s["hq"], s["hk"], s["hk"]), dim=1))
    y, mag = ref.norm_rope(q, cpu(s["qg"]), 1e-6, 0.0, cpu(s["table"]), cpu(s["pos"]), False)
    ref.check_bf16(cpu(s["q_out"]), y, ref.norm_error(mag), "q")
    y, mag = ref.norm_rope(k, cpu(s["kg"]), 1e-6, 0.0, cpu(s["table"]), cpu(s["pos"]), False)
    for got, x, err in ((s["out"][0], y, ref.norm_error(mag)),
                        (s["out"][1], v.double(), torch.zeros_like(v.double()))):
        # half an e4m3 step of the row's scale (2^-4 relative, and half the
        # smallest step, scale * 2^-10), then half a bf16 step
        scale = ref.row_scale(x, INF)[..., None]
        e4 = x.abs() * 2.0 ** -4 + scale * 2.0 ** -10 + 2 * err + 8 * ref.U * x.abs()
        ref.check_bf16(cpu(got), x, e4, "read back")


def test_a_step_together(rrf):
    s = step_problem(rrf, 1)
    step(rrf, s)
    check_step(s)


def test_captured_and_replayed(rrf):
    """Two graphs of the step on their own buffers, replayed in turn with new
    inputs, on streams other than the one the tensors were made on."""
    states = [step_problem(rrf, n) for n in (2, 3)]
    for s in states:
        step(rrf, s)
    torch.cuda.synchronize()
    graphs = []
    for s in states:
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            step(rrf, s)
        graphs.append(graph)
    other = torch.cuda.Stream()
    for turn in range(2):
        for s in states:
            s["a"].view(torch.uint8).copy_(s["a"].view(torch.uint8).flip(0))
        torch.cuda.synchronize()
        graphs[0].replay()
        with torch.cuda.stream(other):
            graphs[1].replay()
        torch.cuda.synchronize()
        for s in states:
            check_step(s)
            got = [t.clone() for t in (s["q_out"], *s["out"])]
            step(rrf, s)
            torch.cuda.synchronize()
            assert all(torch.equal(a, b) for a, b in zip(got, (s["q_out"], *s["out"])))


def test_current_stream_is_used(rrf):
    s = step_problem(rrf, 4)
    step(rrf, s)
    torch.cuda.synchronize()
    want = [t.clone() for t in (s["q_out"], *s["out"])]
    for t in (s["q_out"], *s["out"], s["qkv"]):
        t.zero_()
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        torch.cuda._sleep(2_000_000)
        step(rrf, s)
    assert bool((s["q_out"] == 0).all())  # queued behind the sleep on `side`
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(want, (s["q_out"], *s["out"])))


def test_two_streams_at_once(rrf):
    """Calls that overlap on the GPU share nothing."""
    states = [step_problem(rrf, 20 + n, tokens=512, hidden=1024) for n in range(2)]
    streams = [torch.cuda.Stream() for _ in states]
    torch.cuda.synchronize()
    for _ in range(20):
        for s, stream in zip(states, streams):
            with torch.cuda.stream(stream):
                step(rrf, s)
    torch.cuda.synchronize()
    for s in states:
        check_step(s)


def test_refusals_of_tensors(rrf):
    """Each refusal names its tensor, and nothing is written."""
    q, k, v, qg, kg, table, pos = problem(2, 6, 2, 1, 64, 64)
    cache = new_cache(gen(1), 4, 16, 1, 64)
    before = clone_cache(cache)
    slots = torch.arange(6, device="cuda")
    args = dict(q=q, k=k, v=v, q_gamma=qg, k_gamma=kg, eps=1e-6, weight_offset=0.0, cos_sin=table,
                positions=pos, slots=slots, k_cache=cache[0], k_scales=cache[1],
                v_cache=cache[2], v_scales=cache[3])
    wide = torch.zeros((6, 2, 128), dtype=torch.bfloat16, device="cuda")
    for name, bad in [("q", q.float()), ("q", q[:, 0]), ("k", k[:5]), ("k", k[..., :32]),
                      ("v", v.transpose(1, 2).contiguous().transpose(1, 2)[:, :, :1]),
                      ("q", wide[..., ::2]), ("q_gamma", qg[:32]), ("k_gamma", kg.float()),
                      ("cos_sin", table.double()), ("cos_sin", table[:, ::2]),
                      ("positions", pos.int()), ("positions", pos[:5]), ("positions", None),
                      ("slots", slots.int()), ("slots", slots[:5]), ("slots", slots.cpu()),
                      ("k_cache", cache[0].view(torch.uint8)), ("k_cache", cache[0][:, :8]),
                      ("v_cache", cache[2].transpose(1, 3)), ("k_scales", cache[1].double()),
                      ("v_scales", cache[3][:3]), ("q", None), ("k_cache", 3)]:
        with pytest.raises(ValueError, match="cache|scales" if name[1:] in ("_cache", "_scales")
                           else name):
            rrf.rrf_qk_norm_rope_kv_cache_fp8(**{**args, name: bad})
    with pytest.raises(RuntimeError, match="ambiguous"):  # (no truth value)
        rrf.rrf_qk_norm_rope_kv_cache_fp8(**args, interleaved=torch.zeros(2))
    with pytest.raises(rrf.RrfError) as e:
        rrf.rrf_qk_norm_rope_kv_cache_fp8(**{**args, "eps": -1.0})
    assert e.value.status == rrf.Status.ERR_VALUE
    with pytest.raises(rrf.RrfError) as e:  # heads on one another
        rrf.rrf_qk_norm_rope_kv_cache_fp8(**args, q_out=q[:, :1].expand(6, 2, 64))
    assert e.value.status == rrf.Status.ERR_ALIAS
    for a, b in zip(clone_cache(cache), before):
        assert torch.equal(a, b)


def test_parameters_need_no_grad(rrf):
    """A gamma that is a parameter: refused where autograd records, and the
    same result as its values under no_grad and in inference mode."""
    q, k, v, qg, kg, table, pos = problem(3, 5, 2, 1, 64, 64)
    w = torch.nn.Parameter(qg.clone())
    want = rrf.rrf_qk_norm_rope(q, k, qg, kg, 1e-6, 0.0, table, pos)
    with pytest.raises(ValueError, match="q_gamma must be .*require grad"):
        rrf.rrf_qk_norm_rope(q, k, w, kg, 1e-6, 0.0, table, pos)
    for mode in (torch.no_grad, torch.inference_mode):
        with mode():
            got = rrf.rrf_qk_norm_rope(q, k, w, kg, 1e-6, 0.0, table, pos)
        assert all(torch.equal(x, y) for x, y in zip(got, want))
    cache = new_cache(gen(1), 4, 16, 1, 64)
    cache[1].requires_grad_()
    with pytest.raises(ValueError, match="k_scales must be .*require grad"):
        rrf.rrf_kv_cache_write_fp8(k, v, pos[:5] % 64, *cache)


def test_written_tensors_count_a_version(rrf):
    """Autograd learns of a tensor that a call wrote: a backward pass that had
    saved it is refused, as after any write in place.  The inputs' versions
    stay."""
    q, k, v, qg, kg, table, pos = (x.contiguous() for x in problem(3, 5, 2, 1, 64, 64))
    cache = new_cache(gen(1), 4, 16, 1, 64)
    slots = torch.arange(5, device="cuda")
    qo, ko = torch.empty_like(q), torch.empty_like(k)
    starts = torch.tensor([0, 5], dtype=torch.int32, device="cuda")
    block = torch.zeros((1, 1), dtype=torch.int32, device="cuda")
    ins = (q, k, v, qg, kg, table, pos, slots, starts, block)
    for call, outs in (
            (lambda: rrf.rrf_qk_norm_rope(q, k, qg, kg, 1e-6, 0.0, table, pos, q_out=qo,
                                          k_out=ko), (qo, ko)),
            (lambda: rrf.rrf_kv_cache_write_fp8(k, v, slots, *cache), cache),
            (lambda: rrf.rrf_qk_norm_rope_kv_cache_fp8(q, k, v, qg, kg, 1e-6, 0.0, table, pos,
                                                       slots, *cache, q_out=qo), (qo, *cache)),
            (lambda: rrf.rrf_kv_cache_read_fp8(*cache, block, starts, qo[:, :1].contiguous(),
                                               ko), (ko,))):
        before, kept = [t._version for t in outs], [t._version for t in ins]
        call()
        assert all(t._version > n for t, n in zip(outs, before))
        assert [t._version for t in ins] == kept
    x = torch.ones(q.shape, device="cuda", requires_grad=True)
    y = x * q
    rrf.rrf_qk_norm_rope(q, k, qg, kg, 1e-6, 0.0, table, pos, q_out=q)
    with pytest.raises(RuntimeError, match="modified by an inplace operation"):
        y.sum().backward()
    with torch.inference_mode():  # (its tensors count none)
        mine = torch.empty_like(q)
        rrf.rrf_qk_norm_rope(q, k, qg, kg, 1e-6, 0.0, table, pos, q_out=mine)


def test_empty_calls(rrf):
    q, k, v, qg, kg, table, pos = problem(1, 1, 2, 1, 64, 64)
    cache = new_cache(gen(1), 2, 16, 1, 64)
    before = clone_cache(cache)
    none = torch.empty(0, dtype=torch.int64, device="cuda")
    qo, ko = rrf.rrf_qk_norm_rope(q[:0], k[:0], qg, kg, 1e-6, 0.0, table, none)
    assert qo.shape == (0, 2, 64) and ko.shape == (0, 1, 64)
    rrf.rrf_kv_cache_write_fp8(k[:0], v[:0], none, *cache)
    assert rrf.rrf_qk_norm_rope_kv_cache_fp8(q[:0], k[:0], v[:0], qg, kg, 1e-6, 0.0, table, none,
                                             none, *cache).shape == (0, 2, 64)
    out = [torch.full((2, 1, 64), 3.0, dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    table0 = torch.empty((0, 3), dtype=torch.int32, device="cuda")
    rrf.rrf_kv_cache_read_fp8(*cache, table0, torch.zeros(1, device="cuda").int(), *out)
    assert bool((out[0] == 3).all())
    # a batch that is padding alone
    rrf.rrf_kv_cache_write_fp8(k, v, torch.tensor([-1], device="cuda"), *cache)
    for a, b in zip(clone_cache(cache), before):
        assert torch.equal(a, b)


_CHECKED = r'''
import sys
sys.path[:0] = [ROOT, HERE]
import reduce_rmsnorm_fp8_b200 as rrf
import test_gpu_heads as t
assert rrf.LIB_PATH.endswith("librrf_debug.so"), rrf.LIB_PATH
rrf.rrf_device_error(clear=True)
for shape in t.SHAPES:
    t.test_norm_rope(rrf, shape, True)
    t.test_fused(rrf, shape, False, "hnd")
    t.test_cache_write(rrf, shape, 5, "gaps")
for lens in ([1], [0, 5, 0, 17], [33, 1, 70, 2], [3] * 300):
    t.test_read(rrf, lens, 7, 1, 16, "hnd")
    t.test_read(rrf, lens, 64, 8, 128, "gaps")
t.test_in_place_and_head_major(rrf)
assert rrf.rrf_device_error() == 0
print("checked build clean")
'''


def test_bounds_checking_build(rrf):
    """The bounds-checking build runs the same cases with a clear error word."""
    import os
    import subprocess
    import sys
    from reduce_rmsnorm_fp8_b200 import build
    build.build(debug=True)
    here = os.path.dirname(os.path.abspath(__file__))
    root = os.path.dirname(here)
    p = subprocess.run([sys.executable, "-c", f"ROOT = {root!r}\nHERE = {here!r}\n" + _CHECKED],
                       env=dict(os.environ, RRF_DEBUG_LIBRARY="1"), cwd=root,
                       capture_output=True, text=True, timeout=600)
    assert p.returncode == 0 and "checked build clean" in p.stdout, (p.stdout + p.stderr)[-4000:]
