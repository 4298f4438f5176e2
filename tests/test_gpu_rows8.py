"""8-bit rows on the GPU against the formula in 64 bits, bit for bit.

The scale is the 64-bit quotient a / 127 rounded once to float32 (a is a float32
number, so that is the correctly rounded float32 quotient), the code the whole
number nearest to the 64-bit quotient x / s, half to even: the quotient of two
float32 numbers is either exactly a half or at least 2^-25 of itself away from
it, which 64 bits tell apart.  Restored values are the float32 product of code
and scale, rounded to the type by the CPU.  So nothing here has a tolerance.
"""

import pytest
import torch

pytestmark = pytest.mark.gpu

TYPES = [torch.bfloat16, torch.float16, torch.float32]
GROUPS = [0, 32, 64, 128, 256]


@pytest.fixture(scope="module", autouse=True)
def _built():
    from gptq_qqq_calibration_gb300 import build as b
    b.build()


def formula(x, group):
    """(codes int8, scales float32) of a CPU tensor [n, d]."""
    n, d = x.shape
    width = d if group == 0 else group
    v = torch.nn.functional.pad(x.double(), (0, -d % width)).view(n, -1, width)
    top = v.abs().amax(dim=2)
    s = (top / 127.0).float()
    wide = s[:, :, None].double()
    q = torch.where(wide > 0, torch.round(v / wide).clamp(-127, 127), torch.zeros_like(v))
    bad = ~torch.isfinite(v).all(dim=2)
    q[bad] = 0.0
    s[bad] = float("nan")
    return q.reshape(n, -1)[:, :d].to(torch.int8), s[:, 0] if group == 0 else s


def values(codes, scale, group, dtype):
    n, d = codes.shape
    wide = scale.view(n, -1)
    wide = wide if group == 0 else wide.repeat_interleave(group, dim=1)[:, :d]
    return (codes.float() * wide).to(dtype)


def same(a, b):
    return torch.equal(a.cpu().view(torch.uint8) if a.dtype == torch.int8 else torch.nan_to_num(a.cpu().float(), 7.25),
                       b.view(torch.uint8) if b.dtype == torch.int8 else torch.nan_to_num(b.float(), 7.25))


def make(n, d, dtype, seed, scale=1.0):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn((n, d), generator=g) * scale
    x[:, torch.rand(d, generator=g) < 0.02] *= 20.0
    x[torch.rand(n, generator=g) < 0.1] = 0.0
    return x.to(dtype)


def check(x, group, X=None):
    from gptq_qqq_calibration_gb300 import quantize_rows, restore_rows
    codes, scale = formula(x, group)
    rows = quantize_rows(x.cuda() if X is None else X, group=group)
    assert same(rows.scale, scale) and same(rows.codes, codes)
    for dtype in TYPES:
        assert same(restore_rows(rows, dtype), values(codes, scale, group, dtype))


SIZES = [(1, 1), (1, 8), (3, 7), (2, 31), (5, 33), (4, 256), (3, 257), (7, 520), (1, 1024), (2, 1025), (33, 2564),
         (1, 4096), (600, 264), (513, 1032), (700, 1480), (2, 16384), (2, 16392), (530, 4104), (3, 70000), (1, 69999),
         # rows that join to longer ones, and rows whose ends cut the runs of a restoring lane
         (67, 128), (1001, 64), (4099, 32), (130, 256), (90, 384), (40, 8191), (11, 17), (600, 35), (300, 259),
         (519, 1033), (700, 2049), (1601, 8191), (515, 1990), (2000, 1100)]


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("n,d", SIZES)
def test_sizes(n, d, dtype):
    for group in GROUPS:
        check(make(n, d, dtype, n + d + group), group)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("group", [0, 64])
def test_values_at_the_edges(dtype, group):
    """Halves, NaN, infinities, zeros, the type's largest and smallest numbers."""
    big, tiny = torch.finfo(dtype).max, torch.finfo(dtype).smallest_normal
    sub = torch.finfo(dtype).tiny * torch.finfo(dtype).eps  # the smallest subnormal
    ramp = torch.arange(-128, 128).float()
    rows = [ramp * 0.5 / 127 * 127,             # maximum 64: quotients that end on halves
            (ramp.clamp(-127, 127) + 0.5).clamp(-127, 127), (ramp * 2 + 1).clamp(-254, 254) / 2,
            torch.full((256,), 0.0), torch.full((256,), -0.0), torch.full((256,), big),
            torch.linspace(-big, big, 256, dtype=torch.float64), ramp * tiny, ramp * sub, ramp.clamp(-3, 3) * sub,
            ramp * sub * 3, torch.full((256,), tiny)]
    for bad in (float("nan"), float("inf"), -float("inf")):
        for at in (0, 100, 255):
            r = ramp.clone()
            r[at] = bad
            rows.append(r)
    x = torch.stack([r.double() for r in rows]).to(dtype)
    for width in (256, 255):
        check(x[:, :width].contiguous(), group)
        wide = torch.cat([x[:, :width], torch.zeros((x.shape[0], 1024 - width), dtype=dtype)], 1)
        check(wide, group)  # the row kernel


def test_exact_halves_everywhere():
    """Rows whose scale is a power of two and whose values are all odd halves of it."""
    g = torch.Generator().manual_seed(5)
    k = torch.randint(-127, 127, (40, 1024), generator=g).float() + 0.5
    k[:, 17] = 127.0
    x = k * torch.exp2(torch.randint(-20, 20, (40, 1), generator=g).float())
    for group in (0, 256):
        check(x, group)


def test_near_halves():
    """float32 quotients within a rounding or two of a half."""
    g = torch.Generator().manual_seed(6)
    top = 1.0 + torch.rand((200, 1), generator=g)
    s = (top.double() / 127).float()
    x = ((torch.randint(-127, 127, (200, 1024), generator=g) + 0.5).double() * s.double()).float()
    step = torch.randint(-3, 4, x.shape, generator=g).int()
    x = (x.view(torch.int32) + step).view(torch.float32)
    x[:, :1] = top
    x = x.clamp(-top, top)
    check(x, 0)
    check(x[:, :1023].contiguous(), 0)


@pytest.mark.parametrize("dtype", TYPES)
def test_views_strides_and_alignment(dtype):
    from gptq_qqq_calibration_gb300 import Rows8, restore_rows
    from gptq_qqq_calibration_gb300.rows8 import rows8_quantize, rows8_restore
    for d, ld, at in ((512, 640, 0), (512, 513, 0), (500, 512, 3), (1032, 1040, 8), (1032, 1044, 4), (64, 65, 1)):
        x = make(37, ld, dtype, d + at)
        X = x.cuda()[:, at:at + d] if at + d <= ld else x.cuda()[:, :d]
        xs = X.cpu().contiguous()
        for group in (0, 32, 128):
            codes, scale = formula(xs, group)
            buf = torch.full((37, ld), 77, dtype=torch.int8, device="cuda")
            C = buf[:, at:at + d] if at + d <= ld else buf[:, :d]
            S = torch.empty(scale.shape, device="cuda")
            rows8_quantize(X, group, C, S)
            assert same(C.contiguous(), codes) and same(S, scale)
            kept = torch.ones((37, ld), dtype=torch.bool)
            kept[:, at if at + d <= ld else 0:][:, :d] = False
            assert (buf.cpu()[kept] == 77).all()  # what lies between the rows
            out = torch.full((37, ld), 5.0, dtype=dtype, device="cuda")
            O = out[:, at:at + d] if at + d <= ld else out[:, :d]  # noqa: E741
            rows8_restore(Rows8(C, S, group), O)
            assert same(O.contiguous(), values(codes, scale, group, dtype)) and (out.cpu()[kept] == 5.0).all()
            assert same(restore_rows(Rows8(C, S, group), dtype), values(codes, scale, group, dtype))


def test_leading_shapes_and_empty():
    from gptq_qqq_calibration_gb300 import quantize_rows, restore_rows
    x = make(24, 320, torch.bfloat16, 3)
    rows = quantize_rows(x.cuda().view(2, 3, 4, 320), group=64)
    codes, scale = formula(x, 64)
    assert rows.codes.shape == (2, 3, 4, 320) and rows.scale.shape == (2, 3, 4, 5)
    assert same(rows.codes.view(24, 320), codes) and same(rows.scale.view(24, 5), scale)
    assert restore_rows(rows).shape == (2, 3, 4, 320)
    assert quantize_rows(x.cuda().view(2, 12, 320)).scale.shape == (2, 12)
    none = quantize_rows(torch.empty((0, 320), device="cuda"), group=32)
    assert none.codes.shape == (0, 320) and none.scale.shape == (0, 10)
    assert restore_rows(none).shape == (0, 320)
    # row by row: the same bits
    for r in (0, 7, 23):
        one = quantize_rows(x[r:r + 1].cuda())
        assert same(one.codes, formula(x, 0)[0][r:r + 1])


@pytest.mark.parametrize("n,d", [(270000, 16384), (33600000, 128), (530003, 8191)])
def test_past_32_bit_offsets(n, d):
    """More than 2^32 codes: rows at the far end, whole and in groups; long, joined and odd ones."""
    from gptq_qqq_calibration_gb300 import quantize_rows, restore_rows
    g = torch.Generator(device="cuda").manual_seed(1)
    X = torch.empty((n, d), dtype=torch.bfloat16, device="cuda")
    for a in range(0, n, 30000):
        X[a:a + 30000] = torch.randn((min(30000, n - a), d), generator=g, device="cuda").bfloat16()
    at = [0, 131071, 131072, 262143, 262144, n - 1]
    for group in (0, 128):
        rows = quantize_rows(X, group=group)
        codes, scale = formula(X[at].cpu(), group)
        assert same(rows.codes[at], codes) and same(rows.scale[at], scale)
        back = restore_rows(rows)
        assert same(back[at], values(codes, scale, group, torch.bfloat16))
        del rows, back


def test_streams_and_graphs():
    from gptq_qqq_calibration_gb300 import quantize_rows, restore_rows
    xs = [make(300, 1000 + 8 * k, torch.float16, k) for k in range(4)]
    streams = [torch.cuda.Stream() for _ in xs]
    dev = [x.cuda() for x in xs]
    torch.cuda.synchronize()
    got = [quantize_rows(x, group=64, stream=s) for x, s in zip(dev, streams)]
    back = [restore_rows(r, torch.float16, stream=s) for r, s in zip(got, streams)]
    torch.cuda.synchronize()
    for x, r, b in zip(xs, got, back):
        codes, scale = formula(x, 64)
        assert same(r.codes, codes) and same(r.scale, scale) and same(b, values(codes, scale, 64, torch.float16))
    graph = torch.cuda.CUDAGraph()
    X = dev[0].clone()
    with torch.cuda.graph(graph):
        rows = quantize_rows(X)
        out = restore_rows(rows, torch.float16)
    for k in (0, 5):
        X.copy_(make(300, 1000, torch.float16, k))
        graph.replay()
        torch.cuda.synchronize()
        codes, scale = formula(X.cpu(), 0)
        assert same(rows.codes, codes) and same(out, values(codes, scale, 0, torch.float16))


def test_writing_into_saved_tensors_is_noticed():
    from gptq_qqq_calibration_gb300 import quantize_rows
    from gptq_qqq_calibration_gb300.rows8 import rows8_restore
    rows = quantize_rows(make(4, 64, torch.float32, 1).cuda())
    out = torch.zeros((4, 64), device="cuda")
    before = out._version
    rows8_restore(rows, out)
    assert out._version > before


def test_refusals():
    from gptq_qqq_calibration_gb300 import HessError, Rows8, _lib, quantize_rows, restore_rows
    x = make(16, 64, torch.bfloat16, 1)
    X = x.cuda()
    rows = quantize_rows(X)
    for bad in (lambda: quantize_rows(x), lambda: quantize_rows(X.double()), lambda: quantize_rows(X.t()),
                lambda: restore_rows(Rows8(rows.codes, rows.scale[:3])), lambda: restore_rows(rows, torch.float64),
                lambda: restore_rows(Rows8(rows.codes, rows.scale, 32)),
                lambda: restore_rows(Rows8(rows.codes.short(), rows.scale)),
                lambda: restore_rows(rows, out=torch.empty((16, 63), device="cuda"))):
        with pytest.raises(ValueError):
            bad()
    for group in (-1, 7, 16, 512):
        with pytest.raises(HessError):
            quantize_rows(X, group=group)
    lib = _lib.load()
    codes, scale = rows.codes, rows.scale
    args = [X.data_ptr(), 64, 16, 64, 0, 0, codes.data_ptr(), 64, scale.data_ptr(), None]
    hostbuf = torch.zeros(16 * 64, dtype=torch.bfloat16)
    for at, wrong in ((0, None), (0, hostbuf.data_ptr()), (0, X.data_ptr() + 1), (1, 63), (2, -1), (3, 0), (4, 9),
                      (6, None), (6, hostbuf.data_ptr()), (6, X.data_ptr() + 2047), (7, 63), (8, None),
                      (8, scale.data_ptr() + 2), (8, codes.data_ptr()), (8, X.data_ptr() + 2044)):
        bad = list(args)
        bad[at] = wrong
        assert lib.rows8_quantize(*bad) == _lib.HESS_ERR_INVALID, (at, wrong)
    out = torch.empty((16, 64), dtype=torch.bfloat16, device="cuda")
    args = [codes.data_ptr(), 64, scale.data_ptr(), 16, 64, 0, out.data_ptr(), 64, 0, None]
    for at, wrong in ((0, None), (0, hostbuf.data_ptr()), (1, 63), (2, None), (2, scale.data_ptr() + 1), (3, -1),
                      (4, 0), (6, None), (6, out.data_ptr() + 1), (6, codes.data_ptr()), (6, scale.data_ptr()),
                      (7, 63), (8, 9)):
        bad = list(args)
        bad[at] = wrong
        assert lib.rows8_restore(*bad) == _lib.HESS_ERR_INVALID, (at, wrong)
    assert lib.rows8_restore(*args) == _lib.HESS_OK
    torch.cuda.synchronize()
