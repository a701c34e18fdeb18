"""Microscaled 4-bit quantisation and the grouped products against plain
implementations in 64 bits.

Tolerances, from the arithmetic alone: quantisation and dequantisation have
one result. A product's terms (4-bit times 4-bit times two powers of two) are
exact in fp32; accumulating them in fp32 in blocks of at least 32 loses at most
2^-22 of the terms' summed magnitudes per block (half a step of rounding, or a
whole one if it truncates, for the block's own sum and for the running one),
so K/32 + 2 such steps bound it. Rounding to bf16 adds 2^-8 of the value. SwiGLU:
|d silu/dg| <= 1.1, and exp, the division and the products in fp32 lose at most
2^-20 of the result."""

import dataclasses
import random

import pytest
import torch

import sparse_top_mixture_b200 as stm
import workloads
from workloads import CONFIGS, reduced

pytestmark = pytest.mark.gpu

GRID = torch.tensor([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0], dtype=torch.float64)


def ref_quantize(x):
    """(values, scale bytes) of x [rows, K] by the definition, in 64 bits on the CPU."""
    b = x.double().cpu().reshape(-1, 32)
    m = b.abs().amax(1)
    bad = ~torch.isfinite(b).all(1)
    _, e = torch.frexp(torch.where(bad, 1.0, m))
    byte = torch.where(m > 0, (e - 1 - 2 + 127).clamp(min=0), 0)
    unit = torch.ldexp(torch.ones_like(m), byte - 127)
    a = torch.where(bad[:, None], 0.0, b).abs() / unit[:, None]
    d = (a[:, :, None] - GRID).abs()
    near = d == d.amin(2, keepdim=True)
    even = near & (torch.arange(8) % 2 == 0)
    pick = torch.where(even.any(2), even.int().argmax(2), near.int().argmax(2))
    v = torch.where(b < 0, -1.0, 1.0) * GRID[pick] * unit[:, None]
    v[bad], byte[bad] = float("nan"), 255
    rows, K = x.shape
    return v.reshape(rows, K), byte.reshape(rows, K // 32).to(torch.uint8)


def ref_values(q):
    """The values of an Mx4 in 64 bits, on its device."""
    data, K = q.data.long(), q.K
    code = torch.stack((data & 15, data >> 4), -1).reshape(*data.shape[:-1], K)
    grid = torch.cat((GRID, -GRID)).to(data.device)
    s = q.scale[..., : K // 32].long()
    # 2^(s - 127) by its fp64 exponent field (a device's pow is not exact)
    unit = torch.where(s == 255, torch.nan, ((s - 127 + 1023) << 52).view(torch.float64))
    return grid[code] * unit.repeat_interleave(32, -1)


def same(a, b):
    return bool(((a == b) | (a.isnan() & b.isnan())).all())


def _rand(shape, dtype=torch.bfloat16, seed=1, std=1.0):
    return (torch.randn(*shape, generator=torch.Generator().manual_seed(seed)) * std).to(dtype).cuda()


# ---- quantisation -----------------------------------------------------------

@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("rows,K", [(1, 32), (3, 64), (5, 96), (2, 512), (7, 544), (300, 1024), (4, 1056), (33, 7168),
                                    (20000, 32), (1, 32 * 700)])
def test_quantize(rows, K, dtype):
    x = _rand((rows, K), dtype, rows + K)
    x *= torch.exp2(torch.randint(-60, 60, (rows, 1), generator=torch.Generator().manual_seed(3)).float()).cuda().to(dtype)
    q = stm.mx4_quantize(x)
    v, byte = ref_quantize(x)
    assert q.K == K and q.shape == (rows, K)
    assert torch.equal(q.scale[:, : K // 32].cpu(), byte)
    assert int(q.scale[:, K // 32:].sum()) == 0
    assert same(ref_values(q).cpu(), v)
    for out in (torch.float32, torch.bfloat16):
        assert same(stm.mx4_dequantize(q, out).double().cpu(), v.to(out).double())


def test_quantize_the_hard_blocks():
    """Zeros of both signs, infinities, NaN, the smallest and the largest
    magnitudes, exact powers of two, and every tie and its neighbours."""
    half = torch.tensor([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, 7.0])
    ties = torch.cat([half, -half, torch.nextafter(half, torch.tensor(9.0)), -torch.nextafter(half, torch.tensor(0.0))])
    blocks = []
    for scale in (2.0 ** -127, 2.0 ** -120, 1.0, 2.0 ** 20, 2.0 ** 124):
        blocks.append(torch.cat([ties[:16], torch.full((16,), 4.0)]) * scale)
        blocks.append(torch.cat([ties[16:], torch.full((16,), 7.9375)]) * scale)
    blocks += [torch.zeros(32), -torch.zeros(32), torch.full((32,), 2.0 ** -133), torch.full((32,), 2.0 ** -149),
               torch.full((32,), torch.finfo(torch.float32).max)]
    for special in (float("inf"), -float("inf"), float("nan")):
        b = torch.ones(32)
        b[13] = special
        blocks.append(b)
    blocks += [torch.full((32,), 2.0 ** i) for i in range(-130, 128)]
    x32 = torch.stack(blocks)
    for x in (x32, x32.to(torch.bfloat16)):
        q = stm.mx4_quantize(x.reshape(-1, 32).cuda())
        v, byte = ref_quantize(x)
        assert torch.equal(q.scale[:, :1].cpu(), byte)
        assert same(ref_values(q).cpu(), v)


def test_dequantize_every_code_and_scale():
    data = torch.arange(256, dtype=torch.uint8).repeat(256, 1).cuda()          # K = 512
    scale = torch.arange(256, dtype=torch.uint8)[:, None].repeat(1, 16).cuda()
    q = stm.Mx4(data, scale)
    v = ref_values(q).cpu()
    for out in (torch.float32, torch.bfloat16):
        assert same(q.dequantize(out).double().cpu(), v.to(out).double())


def test_the_padding_of_the_longest_rows_is_written():
    """K next to 2^31, where a row's last chunk ends past 32 bits."""
    K = (1 << 31) - 32
    x = torch.ones(1, K, dtype=torch.bfloat16, device="cuda")
    data = torch.empty(1, K // 2, dtype=torch.uint8, device="cuda")
    scale = torch.full((1, 1 << 26), 9, dtype=torch.uint8, device="cuda")
    st = stm.lib().moe_mx4_quantize(1, K, stm.DTYPES["bf16"], x.data_ptr(), data.data_ptr(), scale.data_ptr(),
                                    torch.cuda.current_stream().cuda_stream)
    assert st == 0
    assert bool((scale[0, :-1] == 125).all()) and int(scale[0, -1]) == 0  # 2^-2, and one byte of padding
    assert bool((data == 0x66).all())  # 4 = 1 / 2^-2


def test_quantize_shapes():
    x = _rand((3, 5, 64))
    q = stm.mx4_quantize(x)
    assert q.shape == (3, 5, 64) and q.data.shape == (3, 5, 32) and q.scale.shape == (3, 5, 16)
    assert torch.equal(q.dequantize(), stm.mx4_quantize(x.reshape(15, 64)).dequantize().reshape(3, 5, 64))
    one = stm.mx4_quantize(x[0, 0])
    assert one.shape == (64,) and torch.equal(one.data, q.data[0, 0])
    none = stm.mx4_quantize(x[:0])
    assert none.shape == (0, 5, 64) and none.dequantize().shape == (0, 5, 64)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("T,H,E,k,empty", [(1, 32, 1, 1, 0.0), (1, 7168, 256, 8, 0.0), (37, 544, 6, 3, 0.4),
                                           (300, 2080, 64, 9, 0.2)])
def test_quantize_into_sorted_order(T, H, E, k, empty, dtype):
    p = stm.Problem(T=T, H=H, E=E, k=k, I=32, dtype=dtype)
    g = torch.Generator().manual_seed(T)
    sel = torch.rand(T, E, generator=g).topk(k, 1).indices
    sel[torch.rand(T, k, generator=g) < empty] = -1
    plan = stm.dispatch_slots(p, sel.cuda())
    x = _rand((T, H), p.torch_dtype, 4)
    got, ref = stm.mx4_permute_rows(p, x, plan), stm.mx4_quantize(stm.permute_rows(p, x, plan))
    assert torch.equal(got.data, ref.data) and torch.equal(got.scale, ref.scale)


# ---- products ---------------------------------------------------------------

def _offsets(rows, E, seed, kind="spread"):
    """Segment table [E+1] over `rows` rows; "short" leaves rows on both ends outside."""
    g = torch.Generator().manual_seed(seed)
    if kind == "one":
        off = torch.zeros(E + 1, dtype=torch.int32)
        off[E // 2 + 1:] = rows
        return off
    cut = torch.randint(0, rows + 1, (E + 1,), generator=g).sort().values.int()
    if kind != "short":
        cut[0], cut[E] = 0, rows
    return cut


def _operands(rows, E, N, K, seed):
    a, w = stm.mx4_quantize(_rand((rows, K), seed=seed)), stm.mx4_quantize(_rand((E, N, K), seed=seed + 1, std=K ** -0.5))
    return a, w


def _product(a, w, off):
    """(product, summed magnitudes) in 64 bits, rows outside the segments NaN."""
    rows, N = a.data.shape[0], w.data.shape[1]
    y = torch.full((rows, N), float("nan"), dtype=torch.float64, device="cuda")
    mag = torch.zeros_like(y)
    av = ref_values(a)
    for e, (lo, hi) in enumerate(zip(off[:-1].tolist(), off[1:].tolist())):
        if hi > lo:
            we = ref_values(stm.Mx4(w.data[e], w.scale[e]))
            y[lo:hi], mag[lo:hi] = av[lo:hi] @ we.T, av[lo:hi].abs() @ we.abs().T
    return y, mag


def _steps(K):
    return (K / 32 + 2) * 2.0 ** -22


# rows, E, N, K, kind: single values of everything; odd N and K tails (32 mod 64, 64 mod 256, beyond one scale
# vector); segments that start anywhere; one to three units per tile, one to many tiles per CTA; many empty experts
PRODUCTS = [(1, 1, 8, 32, "one"), (3, 4, 40, 64, "spread"), (31, 2, 72, 96, "spread"), (130, 2, 200, 320, "spread"),
            (129, 1, 64, 256, "one"), (257, 8, 264, 544, "spread"), (128, 256, 64, 1056, "spread"),
            (500, 5, 1096, 736, "short"), (1500, 3, 1096, 1056, "spread"), (3000, 3, 1096, 512, "spread"),
            (20000, 7, 648, 288, "spread"), (64, 16, 7168, 2048, "spread"), (40, 3, 512, 7168, "short"),
            (2048, 4, 2048, 768, "spread"), (90, 9, 96, 160, "one")]


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("rows,E,N,K,kind", PRODUCTS)
def test_grouped_matmul(rows, E, N, K, kind, dtype):
    a, w = _operands(rows, E, N, K, seed=rows + K)
    off = _offsets(rows, E, rows + N, kind)
    ws = torch.zeros(256, dtype=torch.uint8, device="cuda")
    got = stm.mx4_grouped_matmul(a, w, off.cuda(), dtype, ws=ws)
    assert stm.read_device_error(ws) == 0
    ref, mag = _product(a, w, off)
    used = slice(int(off[0]), int(off[E]))
    bound = _steps(K) * mag + (2.0 ** -8 * ref.abs() if dtype == torch.bfloat16 else 0)
    assert bool(((got.double() - ref).abs() <= bound)[used].all())


@pytest.mark.parametrize("rows,E,I,H,kind", [(1, 1, 32, 32, "one"), (3, 4, 64, 64, "spread"),
                                             (130, 2, 96, 320, "spread"), (257, 8, 160, 544, "spread"),
                                             (8, 128, 768, 2048, "spread"), (500, 5, 544, 736, "short"),
                                             (3000, 3, 544, 512, "spread"), (20000, 7, 352, 288, "spread"),
                                             (2048, 4, 1408, 768, "spread")])
def test_grouped_gate_up(rows, E, I, H, kind):
    a, w = _operands(rows, E, 2 * I, H, seed=rows + H)
    off = _offsets(rows, E, rows + I, kind)
    ws = torch.zeros(256, dtype=torch.uint8, device="cuda")
    got = stm.mx4_grouped_gate_up(a, w, off.cuda(), ws=ws)
    y, mag = _product(a, w, off)
    g, u, dg, du = y[:, :I], y[:, I:], _steps(H) * mag[:, :I], _steps(H) * mag[:, I:]
    silu = g * torch.sigmoid(g)
    ref = silu * u
    used = slice(int(off[0]), int(off[E]))
    bound = 1.1 * dg * (u.abs() + du) + silu.abs() * du + (2.0 ** -8 + 2.0 ** -20) * (ref.abs() + 1.1 * dg * u.abs() + silu.abs() * du)
    assert bool(((got.double() - ref).abs() <= bound)[used].all())
    q = stm.mx4_grouped_gate_up(a, w, off.cuda(), quantize=True, ws=ws)
    assert stm.read_device_error(ws) == 0
    want = stm.mx4_quantize(got[used].contiguous())
    assert torch.equal(q.data[used], want.data) and torch.equal(q.scale[used], want.scale)


# Segments of 1, 2, 31 ... 257 rows and of none beside large ones: every fill of a tile of 128 and of 256 rows.
LENGTHS = [0, 1, 2, 31, 32, 33, 0, 96, 97, 127, 128, 129, 160, 255, 256, 257, 384, 385]


def _lengths(rows, E):
    """Segments of LENGTHS and then equal ones, over all rows."""
    n = LENGTHS + [0] * (E - len(LENGTHS))
    rest = rows - sum(LENGTHS)
    for e in range(len(LENGTHS), E):
        n[e] = rest // (E - e)
        rest -= n[e]
    return torch.tensor([0] + n, dtype=torch.int32).cumsum(0).int()


# Both sides of the rule for pairs of CTAs (512 rows an expert and 64 steps a pair), with columns that end inside a
# unit, a tile of three units and 16 bytes, and K that ends inside a step and an MMA
@pytest.mark.parametrize("rows,E,N,K", [(3500, 20, 1096, 2080), (11000, 20, 1096, 2080), (11000, 20, 712, 3232),
                                        (24000, 24, 200, 4128), (40000, 30, 2048, 512)])
def test_segments_of_every_length(rows, E, N, K):
    a, w = _operands(rows, E, N, K, seed=rows + N)
    off = _lengths(rows, E)
    ws = torch.zeros(256, dtype=torch.uint8, device="cuda")
    ref, mag = _product(a, w, off)
    for dtype in (torch.float32, torch.bfloat16):
        got = stm.mx4_grouped_matmul(a, w, off.cuda(), dtype, ws=ws)
        bound = _steps(K) * mag + (2.0 ** -8 * ref.abs() if dtype == torch.bfloat16 else 0)
        assert bool(((got.double() - ref).abs() <= bound).all())
    assert stm.read_device_error(ws) == 0


@pytest.mark.parametrize("rows,E,I,H", [(3500, 20, 544, 2080), (11000, 20, 544, 2080), (24000, 24, 96, 4128),
                                        (40000, 30, 1024, 512)])
def test_gate_up_of_segments_of_every_length(rows, E, I, H):
    a, w = _operands(rows, E, 2 * I, H, seed=rows + I)
    off = _lengths(rows, E)
    ws = torch.zeros(256, dtype=torch.uint8, device="cuda")
    got = stm.mx4_grouped_gate_up(a, w, off.cuda(), ws=ws)
    y, mag = _product(a, w, off)
    g, u, dg, du = y[:, :I], y[:, I:], _steps(H) * mag[:, :I], _steps(H) * mag[:, I:]
    silu = g * torch.sigmoid(g)
    ref = silu * u
    slack = 1.1 * dg * (u.abs() + du) + silu.abs() * du
    assert bool(((got.double() - ref).abs() <= slack + (2.0 ** -8 + 2.0 ** -20) * (ref.abs() + slack)).all())
    q = stm.mx4_grouped_gate_up(a, w, off.cuda(), quantize=True, ws=ws)
    want = stm.mx4_quantize(got)
    assert torch.equal(q.data, want.data) and torch.equal(q.scale, want.scale)
    assert stm.read_device_error(ws) == 0


@pytest.mark.parametrize("seed", range(12))
def test_random_products(seed):
    r = random.Random(seed)
    E = r.choice([1, 3, 8, 60, 128, 256])
    N, K = 8 * r.randint(1, 160), 32 * r.randint(1, 70)
    rows = int(2 ** r.uniform(0, 14))
    a, w = _operands(rows, E, N, K, seed=100 + seed)
    off = _offsets(rows, E, seed, r.choice(["spread", "short", "one"]))
    got = stm.mx4_grouped_matmul(a, w, off.cuda(), torch.float32)
    ref, mag = _product(a, w, off)
    used = slice(int(off[0]), int(off[E]))
    assert bool(((got.double() - ref).abs() <= _steps(K) * mag)[used].all())
    I = 32 * r.randint(1, 30)
    a, w = _operands(rows, E, 2 * I, K, seed=200 + seed)
    got = stm.mx4_grouped_gate_up(a, w, off.cuda())
    y, mag = _product(a, w, off)
    g, u, dg, du = y[:, :I], y[:, I:], _steps(K) * mag[:, :I], _steps(K) * mag[:, I:]
    silu = g * torch.sigmoid(g)
    slack = 1.1 * dg * (u.abs() + du) + silu.abs() * du
    bound = slack + (2.0 ** -8 + 2.0 ** -20) * ((silu * u).abs() + slack)
    assert bool(((got.double() - silu * u).abs() <= bound)[used].all())


def test_swiglu_far_from_zero():
    """Gates of large magnitude on both sides, zeros, and products that overflow: as the formula in fp32 has them."""
    values = torch.tensor([0.0, -0.0, 1e-30, -1e-30, 1.0, -1.0, 20.0, -20.0, 87.0, -87.0, -88.5, 89.0, -104.0, 3e4, -3e4,
                           1e30, -1e30, 3e38, -3e38])
    # one row whose products with W are exactly the values: x = e_0 in the first block of 32
    rows, I, H = 1, 32, 32
    x = torch.zeros(rows, H)
    x[0, 0] = 1.0
    for gate in values.tolist():
        q = stm.mx4_quantize(torch.full((1, 32), gate).cuda()).dequantize(torch.float32)[0, 0].double().cpu()
        wt = torch.zeros(1, 2 * I, H)
        wt[0, :I, 0], wt[0, I:, 0] = gate, 1.0
        off = torch.tensor([0, 1], dtype=torch.int32, device="cuda")
        got = stm.mx4_grouped_gate_up(stm.mx4_quantize(x.cuda()), stm.mx4_quantize(wt.cuda()), off).double().cpu()
        ref = q * torch.sigmoid(q)
        assert bool(((got - ref).abs() <= (2.0 ** -8 + 2.0 ** -20) * ref.abs() + 2.0 ** -119 * q.abs() + 2.0 ** -133).all()), gate


def test_swiglu_where_the_gate_almost_vanishes():
    """Gates so negative that 1 / (1 + e^-g) is subnormal in fp32 while silu(g), or its product with a large up value,
    is not. Off by 2^-20 of the value (see above) and by half a subnormal step of the sigmoid, 2^-150, times |g|; the
    product is rounded to bf16."""
    gates = torch.tensor([-80.0, -86.5, -87.0, -87.25, -87.5, -88.0, -88.5, -88.75, -89.0, -90.0, -92.5, -95.0, -97.25,
                          -100.0, -104.0, -110.5, -112.0, -120.5, -127.0, -130.0, -131.0, -132.0, -133.0, -133.5, -140.0,
                          -200.0, 0.5, 87.5, 88.5, 100.0, 133.5, 200.0], dtype=torch.float64)
    # row 0 of A has a one in the first place of each block of 32, and W's row n the bits of gate n, one to a block
    I, bits = 32, [2.0 ** i for i in range(7, -3, -1)]
    K = 32 * len(bits)
    x, wt = torch.zeros(1, K), torch.zeros(1, 2 * I, K)
    x[0, ::32] = 1.0
    for n, gate in enumerate(gates.tolist()):
        left = abs(gate)
        for i, bit in enumerate(bits):
            if left >= bit:
                wt[0, n, 32 * i] = bit if gate > 0 else -bit
                left -= bit
        assert left == 0
    off = torch.tensor([0, 1], dtype=torch.int32, device="cuda")
    for up in (1.0, 2.0 ** 60, 2.0 ** 100, 2.0 ** 118):
        wt[0, I:, 0] = up
        got = stm.mx4_grouped_gate_up(stm.mx4_quantize(x.cuda()), stm.mx4_quantize(wt.cuda()), off)[0].double().cpu()
        ref = gates * torch.sigmoid(gates) * up
        bound = (2.0 ** -8 + 2.0 ** -20) * ref.abs() + 2.0 ** -150 * gates.abs() * up + 2.0 ** -133
        assert bool(((got - ref).abs() <= bound).all()), gates[(got - ref).abs() > bound]


def test_a_product_longer_than_a_wait():
    """A launch of pairs that runs for seconds, longer than any one of its bounded waits. Codes with scales of 1 are
    multiples of 1/2, and a sum of 393216 of their products (at most 36 each, of either sign) stays far below 2^22, so
    that fp32 holds every partial sum exactly."""
    rows, N, K = 98304, 98304, 393216
    g = torch.Generator(device="cuda").manual_seed(1)

    def codes(*lead):
        return stm.Mx4(torch.randint(0, 256, (*lead, K // 2), dtype=torch.uint8, device="cuda", generator=g),
                       torch.full((*lead, K // 32), 127, dtype=torch.uint8, device="cuda"))

    a, w = codes(rows), codes(1, N)
    off = torch.tensor([0, rows], dtype=torch.int32, device="cuda")
    ws = torch.zeros(256, dtype=torch.uint8, device="cuda")
    y = stm.mx4_grouped_matmul(a, w, off, ws=ws)
    assert stm.read_device_error(ws) == 0
    i = torch.cat((torch.arange(0, rows, 1531), torch.arange(rows - 256, rows, 5))).cuda()
    j = torch.cat((torch.arange(0, N, 769), torch.arange(N - 200, N, 7))).cuda()
    ref = ref_values(stm.Mx4(a.data[i], a.scale[i])) @ ref_values(stm.Mx4(w.data[0, j], w.scale[0, j])).T
    assert float(ref.abs().max()) < 2 ** 20
    assert torch.equal(y[i][:, j], ref.to(torch.bfloat16))


@pytest.mark.parametrize("gate_up", [False, True])
def test_a_pair_uses_the_scales_of_its_own_rows(gate_up):
    """Scales that change in every block, from launch to launch and stage to stage: a word that a CTA of a pair copied
    before it was written would show. Codes (multiples of 1/2 up to 6) and scales of 1, 2 and 4 make every partial sum
    of 4096 products a multiple of 1/4 below 4096 * 36 * 16 < 2^22: exact in fp32 in any order."""
    rows, N, K = 4096, 4096, 4096
    off = torch.tensor([0, rows], dtype=torch.int32, device="cuda")
    g = torch.Generator(device="cuda").manual_seed(3)
    a = stm.Mx4(torch.randint(0, 256, (rows, K // 2), dtype=torch.uint8, device="cuda", generator=g),
                torch.empty(rows, K // 32, dtype=torch.uint8, device="cuda"))
    w = stm.Mx4(torch.randint(0, 256, (1, N, K // 2), dtype=torch.uint8, device="cuda", generator=g),
                torch.empty(1, N, K // 32, dtype=torch.uint8, device="cuda"))
    for _ in range(6):
        for q in (a, w):
            q.scale.copy_(torch.randint(127, 130, q.scale.shape, dtype=torch.uint8, device="cuda", generator=g))
        ref = ref_values(a) @ ref_values(w)[0].T
        if gate_up:  # SwiGLU of exact gates and ups
            gate, up = ref.chunk(2, 1)
            ref = gate * torch.sigmoid(gate) * up
            # besides the roundings, half a subnormal step of the sigmoid (2^-150) times gate and up: at gate -104, up
            # 11240 that is 2^-150 * 1168960 = 8.2e-40, more than 2^-130 = 7.3e-40
            bound = (2.0 ** -8 + 2.0 ** -19) * ref.abs() + 2.0 ** -150 * gate.abs() * up.abs() + 2.0 ** -133
            for _ in range(4):
                assert bool(((stm.mx4_grouped_gate_up(a, w, off).double() - ref).abs() <= bound).all())
        else:
            for _ in range(4):
                assert torch.equal(stm.mx4_grouped_matmul(a, w, off, torch.float32).double(), ref)


def test_two_products_at_once_and_replayed():
    """Two streams that run products of different sizes at the same time, and the same from graphs that share a
    workspace."""
    sizes = [(4000, 6, 1096, 1056, 1), (64, 16, 4096, 2048, 2)]
    ws = torch.zeros(256, dtype=torch.uint8, device="cuda")
    runs = []
    for rows, E, N, K, seed in sizes:
        a, w = _operands(rows, E, N, K, seed)
        off = _offsets(rows, E, seed).cuda()
        runs.append((a, w, off, stm.mx4_grouped_matmul(a, w, off, torch.float32, ws=ws)))
    streams = [torch.cuda.Stream() for _ in sizes]
    torch.cuda.synchronize()
    results = [[], []]
    for _ in range(10):
        for i, s in enumerate(streams):
            with torch.cuda.stream(s):
                results[i].append(stm.mx4_grouped_matmul(*runs[i][:3], torch.float32, ws=ws))
    torch.cuda.synchronize()
    for (_, _, _, want), got in zip(runs, results):
        assert all(torch.equal(g, want) for g in got)
    graphs, held = [], []
    for (a, w, off, _), s in zip(runs, streams):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=s):
            held.append(stm.mx4_grouped_matmul(a, w, off, torch.float32, ws=ws))
        graphs.append(g)
    for (a, *_), s in zip(runs, streams):
        a.data.copy_(a.data.flip(0))
        a.scale.copy_(a.scale.flip(0))
    torch.cuda.synchronize()
    for _ in range(3):
        for g, s in zip(graphs, streams):
            with torch.cuda.stream(s):
                g.replay()
    torch.cuda.synchronize()
    for (a, w, off, _), got in zip(runs, held):
        assert torch.equal(got, stm.mx4_grouped_matmul(a, w, off, torch.float32))
    assert stm.read_device_error(ws) == 0


def test_products_are_the_same_every_time():
    a, w = _operands(3000, 6, 704, 1056, 5)
    off = _offsets(3000, 6, 5).cuda()
    first = stm.mx4_grouped_matmul(a, w, off, torch.float32)
    for _ in range(5):
        assert torch.equal(stm.mx4_grouped_matmul(a, w, off, torch.float32), first)


def test_rows_outside_the_segments_are_left_alone():
    rows, E, N, K = 300, 4, 200, 320
    a, w = _operands(rows, E, N, K, 3)
    off = torch.tensor([37, 37, 180, 181, 250], dtype=torch.int32, device="cuda")
    for dt, name in ((torch.float32, 0), (torch.bfloat16, 1)):
        buf = torch.full((rows + 2, N), 7.0, dtype=dt, device="cuda")
        st = stm.lib().moe_mx4_grouped_matmul(rows, E, N, K, name, a.data.data_ptr(), a.scale.data_ptr(),
                                              off.data_ptr(), w.data.data_ptr(), w.scale.data_ptr(), buf[1:].data_ptr(),
                                              None, torch.cuda.current_stream().cuda_stream)
        assert st == 0
        torch.cuda.synchronize()
        out = buf[1:-1]
        assert bool((buf[0] == 7).all() and (buf[-1] == 7).all() and (out[:37] == 7).all() and (out[250:] == 7).all())
        assert torch.equal(out[37:250], stm.mx4_grouped_matmul(a, w, off, dt)[37:250])
    w2 = stm.mx4_quantize(_rand((E, 192, K), seed=9))
    data = torch.full((rows, 48), 9, dtype=torch.uint8, device="cuda")
    scale = torch.full((rows, 16), 9, dtype=torch.uint8, device="cuda")
    st = stm.lib().moe_mx4_grouped_gate_up(rows, E, 96, K, a.data.data_ptr(), a.scale.data_ptr(), off.data_ptr(),
                                           w2.data.data_ptr(), w2.scale.data_ptr(), data.data_ptr(), scale.data_ptr(),
                                           None, torch.cuda.current_stream().cuda_stream)
    assert st == 0
    torch.cuda.synchronize()
    for t in (data, scale):
        assert bool((t[:37] == 9).all() and (t[250:] == 9).all())
    assert int(scale[37:250, 3:].sum()) == 0


def test_nan_scales_stay_in_their_row_and_column():
    rows, E, N, K = 200, 2, 136, 576
    x, wt = _rand((rows, K)), _rand((E, N, K), seed=2)
    x[70, 500], wt[1, 100, 33] = float("nan"), float("inf")
    a, w = stm.mx4_quantize(x), stm.mx4_quantize(wt)
    off = torch.tensor([0, 90, 200], dtype=torch.int32, device="cuda")
    y = stm.mx4_grouped_matmul(a, w, off, torch.float32)
    want = torch.zeros(rows, N, dtype=torch.bool, device="cuda")
    want[70], want[90:, 100] = True, True
    assert torch.equal(y.isnan(), want)


def test_padding_of_the_scales_is_never_used():
    for rows, N, K in ((40, 72, 96), (130, 200, 544), (9, 64, 32)):
        a, w = _operands(rows, 2, N, K, 8)
        off = torch.tensor([0, rows // 2, rows], dtype=torch.int32, device="cuda")
        want = stm.mx4_grouped_matmul(a, w, off, torch.float32)
        for q in (a, w):
            q.scale[..., K // 32:] = 255
        assert torch.equal(stm.mx4_grouped_matmul(a, w, off, torch.float32), want)
        assert bool(a.dequantize().isfinite().all())


def test_a_malformed_table_is_reported_and_computes_nothing():
    a, w = _operands(100, 3, 64, 64, 1)
    for off in ([0, 50, 40, 100], [0, 10, 20, 101], [-1, 10, 20, 100]):
        ws = torch.zeros(256, dtype=torch.uint8, device="cuda")
        off = torch.tensor(off, dtype=torch.int32, device="cuda")
        stm.mx4_grouped_matmul(a, w, off, ws=ws)
        assert stm.read_device_error(ws) == stm.DEVERR_BAD_EXPERT_ID
        stm.mx4_grouped_gate_up(a, w, off, ws=ws)
        assert stm.read_device_error(ws) == stm.DEVERR_BAD_EXPERT_ID


def test_sizes_beyond_32_bits():
    """Elements and bytes past 2^31 and 2^32, checked at both ends."""
    K = 64
    rows = (1 << 31) // K + 1000
    x = torch.randn(1000, K, device="cuda").bfloat16().repeat(rows // 1000 + 1, 1)[:rows].contiguous()
    q = stm.mx4_quantize(x)
    want = stm.mx4_quantize(x[:1000].contiguous())
    for at in (0, rows // 1000 * 1000 - 1000):
        assert torch.equal(q.data[at:at + 1000], want.data) and torch.equal(q.scale[at:at + 1000], want.scale)
    del x
    back = q.dequantize()
    assert torch.equal(back[-1000 - rows % 1000:][:1000], want.dequantize())
    del q, back
    # a product of more outputs than 2^31
    rows, N = 270000, 8192
    a, w = _operands(1000, 2, N, 32, 1)
    a = stm.Mx4(a.data.repeat(270, 1), a.scale.repeat(270, 1))
    off = torch.tensor([0, 1000, rows], dtype=torch.int32, device="cuda")
    y = stm.mx4_grouped_matmul(a, w, off)
    small = stm.mx4_grouped_matmul(stm.Mx4(a.data[:1000], a.scale[:1000]), stm.Mx4(w.data[1:], w.scale[1:]),
                                   torch.tensor([0, 1000], dtype=torch.int32, device="cuda"))
    assert torch.equal(y[-1000:], small) and torch.equal(y[1000:2000], small)
    del y
    # weights of more than 2^32 bytes
    E, N, K = 256, 16384, 2112
    a, w = _operands(100, 1, N, K, 2)
    big = stm.Mx4(torch.zeros(E, N, K // 2, dtype=torch.uint8, device="cuda"),
                  torch.zeros(E, N, w.scale.shape[-1], dtype=torch.uint8, device="cuda"))
    big.data[E - 1], big.scale[E - 1] = w.data[0], w.scale[0]
    off = torch.zeros(E + 1, dtype=torch.int32, device="cuda")
    off[E] = 100
    got = stm.mx4_grouped_matmul(a, big, off, torch.float32)
    assert torch.equal(got, stm.mx4_grouped_matmul(a, w, off[-2:].clone(), torch.float32))


def test_no_rows_and_no_used_experts():
    a, w = _operands(10, 3, 64, 64, 1)
    off = torch.zeros(4, dtype=torch.int32, device="cuda")
    assert stm.mx4_grouped_matmul(stm.Mx4(a.data[:0], a.scale[:0]), w, off).shape == (0, 64)
    assert stm.mx4_grouped_gate_up(stm.Mx4(a.data[:0], a.scale[:0]), w, off, quantize=True).shape == (0, 32)
    assert stm.mx4_grouped_matmul(a, w, off).shape == (10, 64)  # nothing to compute
    torch.cuda.synchronize()


# ---- the layer --------------------------------------------------------------

LAYERS = {
    "qwen3": reduced(CONFIGS["qwen3_30b_a3b"], T=300, H=320, I=224),
    "zipf": reduced(CONFIGS["deepseek_v2_lite_zipf"], T=512, H=256, I=160, I_shared=272),
    "dsv4": reduced(CONFIGS["dsv4_flash_ablation"], T=384, H=512, I=256, I_shared=256),
    "decode": reduced(CONFIGS["decode_weight_streaming"], T=16, H=1024, I=256, I_shared=256),
    "one_token": reduced(CONFIGS["decode_weight_streaming"], T=1, H=544, I=96, I_shared=64),
}


def _layer(name):
    cfg = LAYERS[name]
    dev = {k: (v.cuda() if v is not None else None) for k, v in workloads.generate(cfg, "cpu").items()}
    p = stm.Problem.from_config(cfg)
    return p, dev, stm.Mx4SparseMoE(p, dev)


@pytest.mark.parametrize("name", list(LAYERS))
def test_layer(name):
    """Each stage of the layer in 64 bits, on the 4-bit values that the stage
    before it produced (a value next to a rounding border may fall on either
    side, so the chain is checked stage by stage)."""
    p, dev, moe = _layer(name)
    x = dev["x"]
    out, rw, sel = moe(x)
    assert moe.read_device_error() == 0
    full = stm.SparseMoE(p, dev)
    out16, rw16, sel16 = full(x)
    assert torch.equal(rw, rw16) and torch.equal(sel, sel16)
    assert torch.equal(moe.forward_counts(), torch.bincount(sel.reshape(-1), minlength=p.E).int())

    plan = stm.dispatch(p, sel)
    off = plan["offsets"]
    rows = stm.mx4_permute_rows(p, x, plan)
    v, _ = ref_quantize(x.cpu())
    pos = plan["pair_pos"].long().reshape(p.T, p.k)
    assert same(ref_values(rows)[pos].cpu(), v[:, None].expand(-1, p.k, -1))
    gu, dn = moe.w["gate_up"], moe.w["down"]
    h = stm.mx4_grouped_gate_up(rows, gu, off, quantize=True)
    y, _ = _product(rows, gu, off.cpu())
    g, u = y[:, : p.I], y[:, p.I:]
    near = torch.linalg.norm(ref_values(h) - g * torch.sigmoid(g) * u) / torch.linalg.norm(g * torch.sigmoid(g) * u)
    assert float(near) <= 0.25  # a 4-bit rounding is off by at most a quarter of a value in [4, 8) / 4 ... 6
    yd, ymag = _product(h, dn, off.cpu())
    shared = torch.zeros(p.T, p.H, dtype=torch.float32, device="cuda")
    if p.shared != "none":
        gamma = torch.sigmoid(x.double() @ dev["shared_gate"].double()).float() if p.shared == "sigmoid_gated" else None
        shared = stm.shared_expert(p, x, dev["shared_gate_up"], dev["shared_down"], gamma)
    ref = (yd[pos] * rw.double()[:, :, None]).sum(1) + shared.double()
    slack = ((_steps(p.I) * ymag[pos] + 2.0 ** -8 * yd[pos].abs()) * rw.double()[:, :, None]).sum(1)
    # (the gate's own fp32 rounding enters the gated shared expert)
    slack = slack + 2.0 ** -8 * ref.abs() + 2.0 ** -16 * shared.double().abs()
    assert bool(((out.double() - ref).abs() <= slack * (1 + 2.0 ** -7)).all())
    # and 4 bits stay near the bf16 layer: W and x each off by up to 1/4 in the worst value, about 0.1 in the mean
    rel = float(torch.linalg.norm(out.double() - out16.double()) / torch.linalg.norm(out16.double()))
    assert rel <= 0.5


def test_layer_in_a_graph_and_in_the_host_pipeline():
    p, dev, moe = _layer("dsv4")
    x = dev["x"].clone()
    g = stm.GraphedForward(moe, x)
    pipe = stm.HostPipeline(moe, depth=2)
    for seed in (5, 6, 7):
        batch = _rand((p.T, p.H), seed=seed)
        x.copy_(batch)
        got = [t.clone() for t in g.replay()]
        want = moe(batch)
        assert all(torch.equal(a, b) for a, b in zip(got, want))
        host_in, host_out = batch.cpu().pin_memory(), torch.empty(p.T, p.H, dtype=torch.bfloat16).pin_memory()
        pipe.submit(host_in, host_out)
        pipe.synchronize()
        assert torch.equal(host_out, want[0].cpu())


@pytest.mark.parametrize("base", [stm.SparseMoE, stm.Mx4SparseMoE])
def test_host_pipeline_of_a_subclass(base):
    """Layers whose class is built from other arguments than a problem and weights."""
    p, dev, moe = _layer("dsv4")

    class Named(base):
        def __init__(self, name):
            super().__init__(p, dev)
            self.name = name

    named = Named("first")
    pipe = stm.HostPipeline(named, depth=3)
    assert pipe.slots[0]["moe"] is named
    assert all(isinstance(s["moe"], base) and s["moe"].ws.data_ptr() != named.ws.data_ptr() for s in pipe.slots[1:])
    want = named(dev["x"])[0].cpu()
    for _ in range(3):
        host_out = torch.empty(p.T, p.H, dtype=torch.bfloat16).pin_memory()
        pipe.submit(dev["x"].cpu().pin_memory(), host_out)
        pipe.synchronize()
        assert torch.equal(host_out, want)


@pytest.mark.parametrize("base", [stm.SparseMoE, stm.Mx4SparseMoE])
def test_host_pipeline_runs_a_subclass_in_every_slot(base):
    """A subclass's forward, on every slot's own workspace, stream and counts."""
    p, dev, _ = _layer("dsv4")

    class Doubled(base):
        def forward(self, x, out=None, *args, **kw):
            out, rw, sel = super().forward(x, out, *args, **kw)
            return out.mul_(2), rw, sel

        __call__ = forward

    moe = Doubled(p, dev)
    want = moe(dev["x"])[0].cpu()
    for graphs in (False, True):
        pipe = stm.HostPipeline(moe, depth=3, graphs=graphs)
        slots = [s["moe"] for s in pipe.slots]
        for get in (lambda m: m.ws.data_ptr(), lambda m: m.forward_counts().data_ptr()):
            assert len({get(m) for m in slots}) == 3
        if moe.aux is not None:
            assert len({m.aux.cuda_stream for m in slots}) == 3
        for _ in range(3):
            host_out = torch.empty(p.T, p.H, dtype=torch.bfloat16).pin_memory()
            pipe.submit(dev["x"].cpu().pin_memory(), host_out)
            pipe.synchronize()
            assert torch.equal(host_out, want)


def test_layer_counts_after_a_replay_are_the_replays():
    p, dev, moe = _layer("dsv4")
    x = dev["x"].clone()
    g = stm.GraphedForward(moe, x)
    moe(dev["x"].flip(1).contiguous())  # an eager forward in between
    _, _, sel = g.replay()
    assert torch.equal(moe.forward_counts(), torch.bincount(sel.reshape(-1), minlength=p.E).int())


def test_layer_without_tokens():
    p, dev, _ = _layer("dsv4")
    p0 = dataclasses.replace(p, T=0)
    moe = stm.Mx4SparseMoE(p0, dev)
    out, rw, sel = moe(dev["x"][:0].contiguous())
    assert out.shape == (0, p.H) and rw.shape == (0, p.k) and sel.shape == (0, p.k)
    assert int(moe.forward_counts().sum()) == 0 and moe.read_device_error() == 0


def test_layer_with_the_balancer_and_given_outputs():
    p, dev, moe = _layer("dsv4")
    bal = stm.BiasBalancer(moe, 1e-3)
    out = torch.empty(p.T, p.H, dtype=torch.bfloat16, device="cuda")
    got, rw, sel = moe(dev["x"], out=out)
    assert got is out
    bal.stash()
    before = dev["bias"].clone()
    bal.update()
    load = torch.bincount(sel.reshape(-1), minlength=p.E).double()
    step = torch.sign(load.mean() - load).float() * 1e-3
    assert torch.allclose(dev["bias"], before + step, atol=1e-7)
    again = stm.Mx4SparseMoE(p, moe.w)  # weights that are 4 bits already
    assert again.w["gate_up"] is moe.w["gate_up"]
    assert torch.equal(again(dev["x"])[1], moe(dev["x"])[1])


def test_trained_rows_then_served_in_4_bits():
    """The operators together: a step of training through permute_rows and
    unpermute_rows, its weights quantised, and the same tokens served."""
    p = stm.Problem(T=64, H=64, E=4, k=2, I=64)
    g = torch.Generator().manual_seed(0)
    x = torch.randn(p.T, p.H, generator=g).bfloat16().cuda()
    gate_w = (torch.randn(p.E, p.H, generator=g) / 8).bfloat16().cuda()
    gu = (torch.randn(p.E, 2 * p.I, p.H, generator=g) / 8).cuda().requires_grad_(True)
    dn = (torch.randn(p.E, p.H, p.I, generator=g) / 8).cuda().requires_grad_(True)
    rw, sel, _ = stm.route(p, x, gate_w)
    plan = stm.dispatch(p, sel)
    off = plan["offsets"].tolist()

    def experts(rows):
        ys = []
        for e in range(p.E):
            gate, up = (rows[off[e]:off[e + 1]].float() @ gu[e].T).chunk(2, 1)
            ys.append((torch.nn.functional.silu(gate) * up) @ dn[e].T)
        return torch.cat(ys)

    out = stm.unpermute_rows(p, experts(stm.permute_rows(p, x, plan)), plan, rw)
    out.float().square().mean().backward()
    assert all(bool(torch.isfinite(t.grad).all()) and float(t.grad.abs().sum()) > 0 for t in (gu, dn))
    with torch.no_grad():
        gu -= 0.1 * gu.grad
        dn -= 0.1 * dn.grad
        plain = stm.unpermute_rows(p, experts(stm.permute_rows(p, x, plan)), plan, rw)
    served, rw4, sel4 = stm.Mx4SparseMoE(p, {"gate_w": gate_w, "gate_up": gu.detach().bfloat16(),
                                             "down": dn.detach().bfloat16()})(x)
    assert torch.equal(sel4, sel) and torch.equal(rw4, rw)
    assert float(torch.linalg.norm(served.float() - plain.float()) / torch.linalg.norm(plain.float())) <= 0.5


def test_refusals():
    x = _rand((4, 64))
    q = stm.mx4_quantize(x)
    w = stm.mx4_quantize(_rand((2, 64, 64)))
    off = torch.tensor([0, 2, 4], dtype=torch.int32, device="cuda")
    short = stm.Mx4(q.data, q.scale[:, :8].contiguous())
    p = stm.Problem(T=4, H=64, E=2, k=1, I=32)
    plan = stm.dispatch(p, torch.zeros(4, 1, dtype=torch.int64, device="cuda"))
    bad = [lambda: stm.mx4_quantize(x.half()), lambda: stm.mx4_quantize(x.cpu()), lambda: stm.mx4_quantize(x[:, :48].contiguous()),
           lambda: stm.mx4_quantize(x.t()), lambda: stm.mx4_quantize(x[0, 0]), lambda: stm.mx4_dequantize(short),
           lambda: stm.mx4_dequantize(q, torch.float16), lambda: stm.mx4_dequantize(q.data),
           lambda: stm.mx4_grouped_matmul(short, w, off), lambda: stm.mx4_grouped_matmul(q, q, off),
           lambda: stm.mx4_grouped_matmul(q, w, off[:2]), lambda: stm.mx4_grouped_matmul(q, w, off.long()),
           lambda: stm.mx4_grouped_matmul(q, w, off, torch.float16),
           lambda: stm.mx4_grouped_matmul(q, w, off, ws=torch.zeros(16, device="cuda")),
           lambda: stm.mx4_grouped_matmul(q, stm.mx4_quantize(_rand((2, 64, 96))), off),
           lambda: stm.mx4_grouped_gate_up(q, stm.mx4_quantize(_rand((2, 96, 64))), off),
           lambda: stm.mx4_permute_rows(p, x.float(), plan),
           lambda: stm.Mx4SparseMoE(stm.Problem(T=4, H=64, E=2, k=1, I=32, dtype="f32"), {}),
           lambda: stm.Mx4SparseMoE(stm.Problem(T=4, H=64, E=2, k=1, I=40), {})]
    p, dev, moe = _layer("dsv4")
    half = dev["x"].half()
    bad += [lambda: moe(half), lambda: moe(dev["x"], out=half), lambda: moe(dev["x"][1:]),
            lambda: moe(dev["x"], events=[None]), lambda: stm.Mx4SparseMoE(p, dev, overlap_shared=True),
            lambda: stm.Mx4SparseMoE(p, {**dev, "down": dev["gate_up"]}),
            lambda: stm.Mx4SparseMoE(p, {**dev, "down": moe.w["gate_up"]}),
            lambda: stm.Mx4SparseMoE(p, {**dev, "bias": None}),
            lambda: stm.Mx4SparseMoE(p, {**dev, "gate_w": dev["gate_w"].cpu()})]
    for i, call in enumerate(bad):
        with pytest.raises(ValueError):
            call()
            pytest.fail(f"call {i} was not refused")
    with pytest.raises(stm.MoeError):  # N not a multiple of 8
        stm.mx4_grouped_matmul(q, stm.mx4_quantize(_rand((2, 60, 64))), off)
