"""Products with 4-bit weights against the definition in 64 bits."""
import numpy as np
import pytest

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def tq():
    from ternary_weight_dp4a_gb300 import build
    from ternary_weight_dp4a_gb300 import tq as m
    build.build()
    return m


class Matrix:
    """Random codes, scales and minima; the values and the sums of magnitudes in 64 bits."""

    def __init__(self, tq, n, k, group, mins, seed):
        import torch
        g = torch.Generator(device="cuda")
        g.manual_seed(seed)
        self.n, self.k, self.group = n, k, group
        self.codes = torch.randint(0, 16, (n, k), generator=g, device="cuda", dtype=torch.uint8)
        self.scales = (0.01 + 0.02 * torch.rand((n, k // group), generator=g, device="cuda")).half()
        self.mins = (self.scales.float() * (4 + 8 * torch.rand(self.scales.shape, generator=g, device="cuda"))).half() if mins else None
        self.dev = tq.pack_q4(self.codes, self.scales, self.mins)

    def product(self, x):
        """(x W^T, a bound of the kernel's error in fp32), both float64."""
        import torch
        s = self.scales.double().repeat_interleave(self.group, 1)
        c = self.codes.double()
        b = 8 * s if self.mins is None else self.mins.double().repeat_interleave(self.group, 1)
        x = x.double()
        y = x @ (s * c - b).T
        # what is added up: s * (c - 8) * x, and (8 s - b) * x where there are minima
        size = x.abs() @ (s * (c - 8).abs()).T
        if self.mins is not None:
            size += x.abs() @ (8 * s - b).abs().T
        # a group: at most 128 + 8 additions in the matrix instructions, which may drop bits below 2^-23 of the
        # largest term of each 16 (so 2 * 8 steps of 2^-23 over a group); the sum of x: 128 additions of
        # 2^-24; the fold: one rounding per group for each of its two terms, the rounded 8 s - b, and the parts of at most
        # 16 warps and 8 CTAs.  All relative to the sum of the magnitudes.
        steps = 16 * 2.0 ** -23 + (128 * (self.mins is not None) + 2 * self.k // self.group + 1 + 16 + 8) * 2.0 ** -24
        return y, steps * size


@pytest.fixture(autouse=True)
def no_wait_has_run_out(tq):
    yield
    assert tq.q4_read_error_word() == 0


def _x(m, k, seed):
    import torch
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return torch.randn((m, k), generator=g, device="cuda").bfloat16()


def _check(got, want, tol):
    bad = ~((got.double() - want).abs() <= tol)
    assert not bad.any(), (int(bad.sum()), float((got.double() - want).abs().max()), float(tol.max()))


SIZES = [(1, 128), (15, 128), (16, 256), (17, 384), (131, 128), (300, 1024), (1000, 5120), (4099, 640), (96, 17408), (33, 32768)]


@pytest.mark.parametrize("mins", [False, True])
@pytest.mark.parametrize("group", [32, 64, 128])
@pytest.mark.parametrize("n,k", SIZES)
def test_gemv(tq, n, k, group, mins):
    import torch
    w = Matrix(tq, n, k, group, mins, n + k + group)
    for m in (1, 2, 5, 8, 9, 16, 17, 31, 64, 65, 130):
        x = _x(m, k, m)
        want, tol = w.product(x)
        _check(tq.q4_gemv(w.dev, x), want, tol)
        got = tq.q4_gemv(w.dev, x, dtype=torch.bfloat16)
        _check(got, want, tol + 2.0 ** -8 * (want.abs() + tol))


@pytest.mark.parametrize("mins", [False, True])
@pytest.mark.parametrize("group", [32, 64, 128])
@pytest.mark.parametrize("n,k", [(1, 128), (17, 384), (131, 128), (1000, 1024), (4099, 640), (96, 17408), (33, 32768)])
def test_gateup(tq, n, k, group, mins):
    gate, up = Matrix(tq, n, k, group, mins, 1), Matrix(tq, n, k, group, mins, 2)
    for m in (1, 3, 8, 9, 16, 17, 50, 64, 65, 200):
        x = _x(m, k, m)
        g, tg = gate.product(x)
        u, tu = up.product(x)
        s = g * g.sigmoid()
        # |silu'| < 1.1; tq_silu and the product: a few roundings of fp32
        tol = 1.1 * tg * (u.abs() + tu) + s.abs() * tu + 2.0 ** -20 * (s * u).abs()
        _check(tq.q4_gateup(gate.dev, up.dev, x), s * u, tol + 2.0 ** -8 * ((s * u).abs() + tol) + 1e-37)


@pytest.mark.parametrize("m", [300, 512, 700])
def test_many_rows(tq, m):
    import torch
    w, up = Matrix(tq, 1111, 1280, 32, True, 3), Matrix(tq, 1111, 1280, 32, True, 4)
    x = _x(m, 1280, m)
    want, tol = w.product(x)
    _check(tq.q4_gemv(w.dev, x), want, tol)
    u, tu = up.product(x)
    s = want * want.sigmoid()
    tol = 1.1 * tol * (u.abs() + tu) + s.abs() * tu + 2.0 ** -20 * (s * u).abs()
    _check(tq.q4_gateup(w.dev, up.dev, x), s * u, tol + 2.0 ** -8 * ((s * u).abs() + tol) + 1e-37)
    assert torch.equal(tq.q4_gemv(w.dev, x), tq.q4_gemv(w.dev, x))          # the same every time


@pytest.mark.parametrize("n,k,group,mins", [(20_001, 1024, 64, True), (19_500, 2048, 32, False), (28_700, 1152, 128, True), (19_456, 1024, 32, True)])
def test_more_tiles_than_run_at_once(tq, n, k, group, mins):
    """The last round's tiles are split along k; sizes with 5, 1, 73 and no tiles in it."""
    w = Matrix(tq, n, k, group, mins, 7)
    for m in (17, 100):
        x = _x(m, k, m)
        want, tol = w.product(x)
        _check(tq.q4_gemv(w.dev, x), want, tol)
    half = n // 2
    gate, up = Matrix(tq, half, k, group, mins, 8), Matrix(tq, half, k, group, mins, 9)
    x = _x(40, k, 3)
    g, tg = gate.product(x)
    u, tu = up.product(x)
    s = g * g.sigmoid()
    tol = 1.1 * tg * (u.abs() + tu) + s.abs() * tu + 2.0 ** -20 * (s * u).abs()     # as test_gateup
    _check(tq.q4_gateup(gate.dev, up.dev, x), s * u, tol + 2.0 ** -8 * ((s * u).abs() + tol) + 1e-37)


def test_packed_layout(tq):
    """include/tq_q4.h's formulas, value by value."""
    n, k, group = 21, 256, 64
    w = Matrix(tq, n, k, group, True, 9)
    words = w.dev.codes.cpu().numpy().view(np.uint32)
    scales, mins = w.dev.scales.cpu().numpy(), w.dev.mins.cpu().numpy()
    codes, per = w.codes.cpu().numpy(), 128 // group
    for i in range(32):
        t, r = divmod(i, 16)
        for j in range(k):
            e = j // 128
            at = (t * (k // 128) + e) * 1024 + (r // 8) * 512 + (r % 8) * 64 + ((j % 32) // 8) * 16 + ((j % 128) // 32) * 4
            got = int(words[at // 4]) >> (4 * ((j % 8) // 2 + 4 * (j % 2))) & 15
            assert got == (codes[i, j] if i < n else 8), (i, j)
        for p in range(k // group):
            e, q = divmod(p, per)
            at = (t * (k // 128) + e) * 16 * per + ((r % 8) * 2 + r // 8) * per + q
            for packed, given in ((scales, w.scales), (mins, w.mins)):
                assert packed[at] == (given[i, p].item() if i < n else 0)
    assert w.dev.nbytes == 32 * k // 2 + 2 * 2 * 32 * (k // group)


@pytest.mark.parametrize("n,k,group,mins", [(500, 5120, 128, False), (70, 17408, 32, True), (5000, 256, 64, True)])
def test_a_row_of_a_packed_step_has_the_bits_that_it_has_alone(tq, n, k, group, mins):
    import torch
    w, up = Matrix(tq, n, k, group, mins, 5), Matrix(tq, n, k, group, mins, 6)
    x = _x(8, k, 7)
    alone = torch.cat([tq.q4_gemv(w.dev, x[r:r + 1]) for r in range(8)])
    h = torch.cat([tq.q4_gateup(w.dev, up.dev, x[r:r + 1]) for r in range(8)])
    for m in range(2, 9):
        assert torch.equal(tq.q4_gemv(w.dev, x[:m]), alone[:m])
        assert torch.equal(tq.q4_gateup(w.dev, up.dev, x[:m]), h[:m])


@pytest.mark.parametrize("m", [1, 8, 12, 40, 100])
def test_nothing_else_is_written(tq, m):
    """Rows of an odd width in the middle of a buffer, at every alignment that is allowed."""
    import torch
    n, k = 77, 256
    w, up = Matrix(tq, n, k, 64, False, 5), Matrix(tq, n, k, 64, False, 6)
    x = _x(m, k, 1)
    for dtype in (torch.float32, torch.bfloat16):
        for shift in (0, 1, 3):
            buf = torch.full((m * n + 64,), 7.0, dtype=dtype, device="cuda")
            y = buf[16 + shift:16 + shift + m * n].view(m, n)
            tq.q4_gemv(w.dev, x, y=y)
            assert torch.equal(y, tq.q4_gemv(w.dev, x, dtype=dtype))
            assert (buf[:16 + shift] == 7).all() and (buf[16 + shift + m * n:] == 7).all()
    buf = torch.full((m * n + 64,), 7.0, dtype=torch.bfloat16, device="cuda")
    h = buf[17:17 + m * n].view(m, n)
    tq.q4_gateup(w.dev, up.dev, x, h=h)
    assert torch.equal(h, tq.q4_gateup(w.dev, up.dev, x)) and (buf[:17] == 7).all() and (buf[17 + m * n:] == 7).all()


@pytest.mark.parametrize("m", [1, 8, 20, 80])
def test_infinities_and_nan_stay_in_their_rows(tq, m):
    import torch
    w = Matrix(tq, 40, 512, 128, True, 5)
    x = _x(m, 512, 1)
    clean = tq.q4_gemv(w.dev, x)
    row = m // 2
    x[row, 100] = float("nan")
    got = tq.q4_gemv(w.dev, x)
    assert got[row].isnan().all()
    keep = torch.arange(m, device="cuda") != row
    assert torch.equal(got[keep], clean[keep])
    x[row, 100] = 0
    x[row, 77] = float("inf")
    got = tq.q4_gemv(w.dev, x)
    assert not got[row].isfinite().any() and torch.equal(got[keep], clean[keep])


@pytest.mark.parametrize("mins", [False, True])
@pytest.mark.parametrize("group", [32, 64, 128])
def test_scales_of_every_size(tq, group, mins):
    """fp16 scales and minima of every exponent and either sign, subnormal ones and zeros among them; and NaN, infinities."""
    import torch
    n, k = 150, 384
    g = torch.Generator(device="cuda")
    g.manual_seed(group + mins)
    codes = torch.randint(0, 16, (n, k), generator=g, device="cuda", dtype=torch.uint8)

    def halves():
        bits = torch.randint(0, 1 << 16, (n, k // group), generator=g, device="cuda", dtype=torch.int32)
        bits = torch.where((bits & 0x7c00) == 0x7c00, bits & 0x83ff, bits)          # no exponent of NaN: subnormal
        return bits.to(torch.int16).view(torch.float16)
    s, b = halves(), halves() if mins else None
    w = tq.pack_q4(codes, s, b)
    sd = s.double().repeat_interleave(group, 1)
    bd = 8 * sd if b is None else b.double().repeat_interleave(group, 1)
    special = s.clone()
    special[20, 1], special[30, 0], special[140, 2] = float("inf"), float("nan"), float("-inf")
    odd = tq.pack_q4(codes, special, b)
    keep = torch.ones(n, dtype=torch.bool, device="cuda")
    keep[[20, 30, 140]] = False
    for m in (1, 9, 17, 64, 100, 192):
        x = _x(m, k, m)
        xd = x.double()
        want = xd @ (sd * codes.double() - bd).T
        size = xd.abs() @ (sd * (codes.double() - 8)).abs().T
        if mins:
            size += xd.abs() @ (8 * sd - bd).abs().T
        # as Matrix.product; with scales in the matrix instructions, 128 values are 16 additions of up to 33/32 of it
        tol = (34 * 2.0 ** -23 + (128 * mins + 2 * k // group + 25) * 2.0 ** -24) * size
        clean = tq.q4_gemv(w, x)
        _check(clean, want, tol)
        got = tq.q4_gemv(odd, x)
        assert torch.equal(got[:, keep], clean[:, keep]) and not got[:, ~keep].isfinite().any()


@pytest.mark.parametrize("m", [64, 80, 192])
@pytest.mark.parametrize("group", [32, 64])
def test_infinities_and_nan_in_wide_calls(tq, group, m):
    import torch
    w = Matrix(tq, 40, 512, group, True, 5)
    x = _x(m, 512, 1)
    clean = tq.q4_gemv(w.dev, x)
    keep = torch.arange(m, device="cuda") != 33
    for bad in ("nan", "inf", "-inf"):
        x[33, 100] = float(bad)
        got = tq.q4_gemv(w.dev, x)
        assert torch.equal(got[keep], clean[keep]) and not got[33].isfinite().any()


def test_offsets_past_32_bits(tq):
    """Packed codes and unpacked ones of more than 2^31 and 2^32 bytes."""
    import torch
    n, k = 140_000, 32768
    codes = torch.zeros((n, k), dtype=torch.uint8, device="cuda")
    codes[-20:] = torch.randint(0, 16, (20, k), device="cuda", dtype=torch.uint8)
    scales = torch.full((n, k // 128), 0.01, device="cuda").half()
    w = tq.pack_q4(codes, scales)
    tail = codes[-20:].double() - 8
    del codes
    for m in (1, 40):
        x = _x(m, k, 1)
        want = x.double() @ tail.T * scales[0, 0].double()
        tol = (16 * 2.0 ** -23 + 600 * 2.0 ** -24) * (x.double().abs() @ tail.abs().T) * scales[0, 0].double()
        _check(tq.q4_gemv(w, x)[:, -20:], want, tol)


def test_outputs_past_32_bits(tq):
    import torch
    n, k, m = 70_001, 128, 32_768
    w = Matrix(tq, n, k, 128, False, 5)
    x = _x(m, k, 1)
    y = torch.empty((m, n), dtype=torch.bfloat16, device="cuda")
    tq.q4_gemv(w.dev, x, y=y)
    for rows in (slice(0, 3), slice(m - 3, m)):
        want, tol = w.product(x[rows])
        _check(y[rows], want, tol + 2.0 ** -8 * (want.abs() + tol))


def test_calls_follow_their_streams_and_replay_in_a_graph(tq):
    import torch
    w, up = Matrix(tq, 300, 1024, 32, True, 5), Matrix(tq, 300, 1024, 32, True, 6)
    xs = {m: _x(m, 1024, m) for m in (1, 8, 40, 200)}
    want = {m: (tq.q4_gemv(w.dev, x), tq.q4_gateup(w.dev, up.dev, x)) for m, x in xs.items()}
    other = torch.cuda.Stream()
    held = {m: torch.zeros_like(x) for m, x in xs.items()}
    torch.cuda.synchronize()
    with torch.cuda.stream(other):
        torch.cuda._sleep(20_000_000)
        for m, x in xs.items():
            held[m].copy_(x)
    got = {m: (tq.q4_gemv(w.dev, held[m], stream=other), tq.q4_gateup(w.dev, up.dev, held[m], stream=other.cuda_stream)) for m in xs}
    other.synchronize()
    for m in xs:
        assert all(torch.equal(a, b) for a, b in zip(got[m], want[m]))
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        out = {m: (tq.q4_gemv(w.dev, held[m]), tq.q4_gateup(w.dev, up.dev, held[m])) for m in xs}
    for m in xs:
        held[m].zero_()
    g.replay()
    for m, x in xs.items():
        held[m].copy_(x)
    g.replay()
    torch.cuda.synchronize()
    for m in xs:
        assert all(torch.equal(a, b) for a, b in zip(out[m], want[m]))


def test_weights_packed_just_before_a_product(tq):
    """The product may start while the work ahead of it in the stream still runs."""
    import torch
    x = _x(1, 5120, 1)
    for seed in range(5):
        w = Matrix(tq, 5120, 5120, 128, False, seed)
        y = tq.q4_gemv(w.dev, x)
        torch.cuda.synchronize()
        assert torch.equal(y, tq.q4_gemv(w.dev, x))
