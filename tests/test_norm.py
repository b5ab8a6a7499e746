"""Root-mean-square norms: refusals on the CPU, results on the GPU against plain float64 forms."""
import pytest
import torch

from _rows import TORCH, half_step
from decode_attention_attn_gb300 import binding, build as lib_build

A = 0x1000000   # an aligned address that no refused call dereferences
FP8 = torch.float8_e4m3fn
# Sums of fp32 squares: each term passes at most E = 16 (its unit) + 8 (units) + 5 + 4 (warp, block) additions, and a
# rounding of its own; terms are positive, so 34 roundings of 2^-24 bound the sum's relative error, half of it the
# root's. The mean, eps, the root and the reciprocal round 4 times, the products with w + o, and w + o, 3 times.
Y_ERR = (34 / 2 + 4 + 3) * 2.0 ** -24


@pytest.fixture(scope="module", autouse=True)
def built():
    lib_build.build()


# ---- CPU: refusals --------------------------------------------------------------------------
def _code(config, args):
    with pytest.raises(binding.DecodeAttnError) as e:
        binding.decode_attn_norm_apply(config, args)
    return e.value.code


def test_apply_refuses_bad_arguments():
    P = 1 << 20

    def call(cfg=(), **kw):
        config = binding.da_norm_config(128, 1e-5, 0.0)
        for k, v in dict(cfg).items():
            setattr(config, k, v)
        row, head = 8 * 128, 128
        args = binding.da_norm_args(A, A + P, A + 2 * P, A + 3 * P, A + 4 * P, A + 5 * P, A + 6 * P, 2, 0, 2, 0, 4, 8,
                                    row, head, row, head, row, head, row, head, row, head, None)
        for k, v in kw.items():
            assert hasattr(args, k)
            setattr(args, k, v)
        return _code(config, args)

    inf, nan = float("inf"), float("nan")
    for cfg, code in ((dict(n=0), -1), (dict(n=32769), -2), (dict(eps=-1.0), -1), (dict(eps=nan), -1),
                      (dict(weight_offset=inf), -1)):
        assert call(cfg) == code, cfg
    assert call(x=None) == -1 and call(out=None, codes=None) == -1
    assert call(residual=None) == -1                       # residual_out without one
    assert call(codes=None) == -1 and call(scales=None) == -1 and call(scaling=0) == -1
    assert call(scaling=4) == -1 and call(scaling=-1) == -1 and call(scaling=3, group=16) == -2
    assert call(scaling=3, group=256) == -2 and call(weight_f32=2) == -1
    assert call(rows=-1) == -1 and call(heads=0) == -1 and call(heads=(1 << 20) + 1) == -2
    assert call(dtype=3) == -2 and call(dtype=-1) == -2
    for name in ("x", "residual", "weight", "residual_out", "out"):
        assert call(**{name: A + 8 * P + 1}) == -1, name
    assert call(scales=A + 8 * P + 2) == -1 and call(weight=A + 8 * P + 2, weight_f32=1) == -1
    # rows on one another, results over inputs and one another
    assert call(out_head_stride=127) == -1 and call(out_row_stride=0) == -1 and call(codes_head_stride=0) == -1
    assert call(residual_out_row_stride=-1024) == -1
    assert call(out=A + 2 * 128 * 3) == -1 and call(out=A, out_row_stride=2048) == -1
    assert call(residual_out=A + P + 16) == -1 and call(codes=A) == -1 and call(codes=A + P) == -1
    assert call(out=A + 3 * P) == -1 and call(codes=A + 4 * P) == -1 and call(out=A + 2 * P) == -1
    assert call(scales=A + 64) == -1 and call(scales=A + 4 * P) == -1 and call(scales=A + 2 * P) == -1
    assert call(scales=A + 5 * P) == -1
    # no rows: nothing is enqueued, no pointer is looked at
    binding.decode_attn_norm_apply(binding.da_norm_config(128, 1e-5, 0.0),
                                   binding.da_norm_args(None, None, None, None, None, None, None, 2, 0, 0, 0, 0, 1))
    with pytest.raises(binding.DecodeAttnError):
        binding._check(binding.lib().decode_attn_norm_apply(None, None), "norm")


def test_wrapper_refuses_bad_tensors():
    with pytest.raises(ValueError):
        binding.RMSNorm(0)
    with pytest.raises(ValueError):
        binding.RMSNorm(32769)
    norm = binding.RMSNorm(64)
    x, w = torch.zeros(3, 64), torch.zeros(64)
    for bad in (torch.zeros(3, 65), torch.zeros(64), torch.zeros(3, 64).double(), torch.zeros(1, 1, 1, 64),
                torch.zeros(64, 3).t()):
        with pytest.raises(ValueError):
            norm.apply(bad)
    for kw in (dict(weight=torch.zeros(65)), dict(weight=w.half()), dict(weight=torch.zeros(128)[::2]),
               dict(residual=torch.zeros(2, 64)), dict(residual=x.half()), dict(residual_out=x),
               dict(out=torch.zeros(3, 128)), dict(out=x.half())):
        with pytest.raises(ValueError):
            norm.apply(x, **kw)
    for kw in (dict(scaling="other"), dict(scaling="group", group=48), dict(scaling="tensor"),
               dict(scales=torch.zeros(2)), dict(scaling="group", scales=torch.zeros(3)), dict(codes=x),
               dict(scaling="tensor", scales=torch.zeros(2)), dict(scales=torch.zeros(3).half()),
               dict(codes=torch.zeros(2, 64, dtype=torch.uint8))):
        with pytest.raises(ValueError):
            norm.quantise(x, w, **kw)
    with pytest.raises(ValueError, match="CUDA"):
        norm.apply(x, w)
    for kw in (dict(x=x.clone().requires_grad_()), dict(weight=w.clone().requires_grad_()),
               dict(residual=x.clone().requires_grad_())):
        with pytest.raises(ValueError, match="gradient"):
            norm.apply(**{"x": x, **kw})


# ---- the plain form -------------------------------------------------------------------------
def plain(x, weight, residual, eps, offset):
    """(y in 64 bits of the stored u, u as it is stored)."""
    u = x if residual is None else (x.float() + residual.float()).to(x.dtype)
    d = u.double()
    y = d / (d.square().mean(-1, keepdim=True) + eps).sqrt()
    if weight is not None:
        y = y * (weight.double() + offset)
    return y, u


def near(got, want, where, least=0.0):
    bound = want.abs() * (half_step(got.dtype) + Y_ERR) + torch.finfo(got.dtype).smallest_normal * half_step(got.dtype) * 2
    err = (got.double() - want).abs()
    assert (err <= bound).all(), (where, float((err / bound).max()))


def check_codes(codes, scale, y, where):
    """Codes within half a step of the quotient by their own scale (2^-4 of it, or half of 2^-9), given that
    y is off by Y_ERR and the quotient rounded."""
    q = (y / scale.double()).clamp(-448, 448)
    err = (codes.view(FP8).double() - q).abs()
    bound = torch.maximum(q.abs() * 2.0 ** -4, torch.full_like(q, 2.0 ** -10)) + q.abs() * (Y_ERR + 2.0 ** -24) * 1.07
    assert (err <= bound).all(), (where, float((err / bound).max()))


def _make(rows, heads, n, dtype, gap=0, shift=0, seed=0, gain=1.0):
    g = torch.Generator().manual_seed(seed + 31 * rows + n)
    wide = torch.zeros(shift + rows * (heads + gap) * n, dtype=TORCH[dtype])
    x = wide[shift:].view(rows, heads + gap, n)
    x.copy_(gain * torch.randn(rows, heads + gap, n, generator=g))
    wide = wide.cuda()
    return wide[shift:].view(rows, heads + gap, n)[:, :heads]


SHAPES = [(1, 1, 1), (3, 1, 7), (5, 3, 64), (64, 40, 128), (9, 2, 100), (2, 1, 4096), (130, 1, 4100), (7, 1, 8192),
          (3, 1, 512), (33, 1, 513), (5, 1, 5119), (2, 1, 16384), (2, 1, 32768), (1, 1, 32767), (4, 1, 24), (11, 5, 272)]


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("rows,heads,n", SHAPES)
@pytest.mark.parametrize("residual,wide_weight,offset", [(False, False, 0.0), (True, False, 1.0), (True, True, 0.0),
                                                         (False, None, 0.0)])
def test_norm(dtype, rows, heads, n, residual, wide_weight, offset):
    x = _make(rows, heads, n, dtype, gain=2.0)
    res = _make(rows, heads, n, dtype, seed=1, gain=3.0) if residual else None
    w = None
    if wide_weight is not None:
        w = (1 - offset + 0.3 * torch.randn(n, generator=torch.Generator().manual_seed(n))).cuda()
        w = w if wide_weight else w.to(TORCH[dtype])
    norm = binding.RMSNorm(n, eps=1e-5, weight_offset=offset)
    want, u = plain(x, w, res, 1e-5, offset)
    got = norm.apply(x, w, residual=res)
    if residual:
        got, total = got
        assert torch.equal(total, u)
    near(got, want, "y")
    for scaling, group in (("row", 0), ("group", 32), ("group", 64), ("group", 128), ("tensor", 0)):
        given = torch.full((1,), 0.0173, device="cuda") if scaling == "tensor" else None
        y32 = torch.empty_like(x) if dtype == "f32" else None
        codes, scales, total = norm.quantise(x, w, residual=res, scaling=scaling, group=group or 128, scales=given, out=y32)
        where = (scaling, group)
        if residual:
            assert torch.equal(total, u), where
        else:
            assert total is None
        if scaling == "tensor":
            each = scales.expand(rows, heads, n)
        else:
            size = n if scaling == "row" else group
            parts = -(-n // size)
            padded = torch.nn.functional.pad(want, (0, parts * size - n)).unflatten(-1, (parts, size))
            most = (padded.abs().amax(-1) / 448).clamp(min=2.0 ** -126)
            assert scales.shape == ((rows, heads) if scaling == "row" else (rows, heads, parts))
            assert ((scales.view(most.shape).double() - most).abs() <= most * (Y_ERR + 2.0 ** -23)).all(), where
            each = scales.view(most.shape)[..., None].expand(-1, -1, -1, size).flatten(-2)[..., :n]
        check_codes(codes, each, want, where)
        if dtype == "f32":
            near(y32, want, where)
            q = (y32 / each).clamp(-448, 448)
            assert torch.equal(codes.view(torch.uint8), q.to(FP8).view(torch.uint8)), where


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("rows,heads,n,gap,shift", [(40, 5, 128, 3, 0), (40, 5, 128, 3, 1), (300, 1, 4096, 1, 8),
                                                    (17, 3, 96, 2, 5), (6, 2, 1000, 1, 16),
                                                    (700, 1, 4099, 0, 8), (700, 1, 1030, 0, 3), (90, 1, 5001, 1, 16)])
def test_strides_alignment_and_in_place(dtype, rows, heads, n, gap, shift):
    """Wide and narrow accesses, results over their inputs, and nothing else written."""
    x = _make(rows, heads, n, dtype, gap, shift)
    res = _make(rows, heads, n, dtype, gap, shift, seed=2)
    w = torch.randn(n, generator=torch.Generator().manual_seed(3)).to(TORCH[dtype]).cuda()
    norm = binding.RMSNorm(n)
    want, u = plain(x, w, res, 1e-6, 0.0)
    got, total = norm.apply(x, w, residual=res)
    assert torch.equal(total, u)
    near(got, want, "apart")
    aligned, _ = norm.apply(x.contiguous(), w, residual=res.contiguous())
    near(aligned, want, "contiguous")
    wide_x, wide_r = x._base, res._base
    others = torch.ones_like(wide_x, dtype=torch.bool)
    others[shift:].view(rows, heads + gap, n)[:, :heads] = False
    x0, r0 = wide_x[others].clone(), wide_r[others].clone()
    again, total = norm.apply(x, w, residual=res, out=x, residual_out=res)
    # (a row's sum goes by how its elements are spread over the threads, which in place may be otherwise)
    assert again is x and total is res and torch.equal(res, u)
    near(x, want, "in place")
    assert torch.equal(wide_x[others], x0) and torch.equal(wide_r[others], r0)
    codes = torch.full((shift + rows * (heads + gap) * n,), 0x55, dtype=torch.uint8, device="cuda")
    view = codes[shift:].view(rows, heads + gap, n)[:, :heads]
    norm.quantise(res, w, codes=view, out=None)
    free, scales, _ = norm.quantise(res.contiguous(), w)
    assert (codes[others] == 0x55).all()
    want, _ = plain(res, w, None, 1e-6, 0.0)
    check_codes(view.contiguous(), norm.quantise(res, w)[1][..., None], want, "strided")
    check_codes(free, scales[..., None], want, "contiguous")


@pytest.mark.gpu
def test_broadcast_rows_and_two_dimensions():
    norm = binding.RMSNorm(256)
    row = torch.randn(1, 256, device="cuda", dtype=torch.bfloat16)
    y = norm.apply(row.expand(70, 256))
    want, _ = plain(row, None, None, 1e-6, 0.0)
    near(y, want.expand(70, 256), "rows")
    res = torch.randn(70, 256, device="cuda", dtype=torch.bfloat16)
    y, u = norm.apply(row.expand(70, 256), residual=res)
    assert torch.equal(u, (row.float() + res.float()).bfloat16())
    heads = torch.randn(7, 256, device="cuda", dtype=torch.float16)[:, None].expand(7, 9, 256)
    near(norm.apply(heads), plain(heads, None, None, 1e-6, 0.0)[0], "heads")
    assert norm.apply(torch.empty(0, 256, device="cuda")).shape == (0, 256)
    codes, scales, u = norm.quantise(torch.empty(0, 3, 256, device="cuda"), scaling="group")
    assert codes.shape == (0, 3, 256) and scales.shape == (0, 3, 2) and u is None


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("n", [128, 100, 4096, 4097])
def test_corner_values(dtype, n):
    """Zeros, infinities, NaN, tiny and huge rows stay in their rows."""
    t = TORCH[dtype]
    x = torch.randn(8, n, generator=torch.Generator().manual_seed(n)).to(t)
    x[1] = 0
    x[2, 5] = float("inf")
    x[3, 7] = float("nan")
    x[4] = x[4] * torch.finfo(t).smallest_normal
    x[5] = x[5] * (2.0 ** 60 if dtype != "f16" else 2.0 ** 12)
    x = x.cuda()
    norm = binding.RMSNorm(n, eps=1e-6)
    want, _ = plain(x, None, None, 1e-6, 0.0)
    y = norm.apply(x)
    plainly = [0, 4, 5, 6, 7]
    near(y[plainly], want[plainly], "rows")
    assert (y[1] == 0).all()
    assert y[2, 5].isnan() and (y[2, :5] == 0).all()       # the others' mean square is infinite
    assert y[3].isnan().all()
    for scaling in ("row", "group", "tensor"):
        given = torch.full((1,), 0.01, device="cuda") if scaling == "tensor" else None
        codes, scales, _ = norm.quantise(x, scaling=scaling, group=32, scales=given)
        v = codes.view(FP8).double()
        assert (v[1] == 0).all() and v[2, 5].isnan() and (v[2, :5] == 0).all() and v[3].isnan().all()
        assert not v[plainly].isnan().any()
        if scaling != "tensor":
            assert (scales[1] == 2.0 ** -126).all() and (scales > 0).all()


@pytest.mark.gpu
def test_zero_eps_and_negative_zero_offset():
    norm = binding.RMSNorm(64, eps=0.0, weight_offset=1.0)
    x = torch.zeros(2, 64, device="cuda")
    x[1] = 1e-18
    w = torch.zeros(64, device="cuda")
    y = norm.apply(x, w)
    assert y[0].isnan().all() and (y[1] - 1).abs().max() < 1e-5


@pytest.mark.gpu
def test_offsets_past_32_bits():
    """Rows more than 2^31 elements apart."""
    n, rows = 64, 3
    big = torch.empty((rows - 1) * ((1 << 31) + 32) + n, dtype=torch.bfloat16, device="cuda")
    x = big.as_strided((rows, n), ((1 << 31) + 32, 1))
    x.copy_(torch.randn(rows, n))
    norm = binding.RMSNorm(n)
    want, _ = plain(x, None, None, 1e-6, 0.0)
    near(norm.apply(x), want, "far")
    norm.apply(x, out=x)
    near(x, want, "far, in place")


@pytest.mark.gpu
def test_many_rows():
    """More rows than blocks of a small grid, the last block part full."""
    x = torch.randn(100003, 1, 64, device="cuda").bfloat16()
    norm = binding.RMSNorm(64)
    near(norm.apply(x), plain(x, None, None, 1e-6, 0.0)[0], "many")
    x = torch.randn(20011, 1024, device="cuda").bfloat16()
    norm = binding.RMSNorm(1024)
    near(norm.apply(x), plain(x, None, None, 1e-6, 0.0)[0], "many")


@pytest.mark.gpu
def test_streams_and_graphs():
    norm = binding.RMSNorm(4096)
    x = torch.randn(5, 4096, device="cuda").bfloat16()
    res, w = torch.randn_like(x), torch.randn(4096, device="cuda").bfloat16()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    y, u = norm.apply(x, w, residual=res, stream=side)
    side.synchronize()
    want, total = plain(x, w, res, 1e-6, 0.0)
    near(y, want, "stream")
    assert torch.equal(u, total)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        codes, scales, u = norm.quantise(x, w, residual=res)
    for seed in range(3):
        x.copy_(torch.randn(5, 4096))
        graph.replay()
        want, total = plain(x, w, res, 1e-6, 0.0)
        assert torch.equal(u, total)
        check_codes(codes, scales[:, None], want, seed)
    # leaves that require a gradient are taken under no_grad
    with torch.no_grad():
        norm.apply(x.clone().requires_grad_(), w)


FAR = [(5, 1, 24), (9, 2, 100), (40, 3, 128), (300, 1, 4096), (3, 1, 513), (700, 1, 4099), (2, 1, 16384)]   # every layout


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("rows,heads,n", FAR)
def test_products_with_the_weight_past_fp32(dtype, rows, heads, n):
    """Rows near the type's end under weights above 1: the products pass fp32, what they are divided by too."""
    x = _make(rows, heads, n, dtype)
    x.clamp_(-4, 4)
    x[::2] *= 2.0 ** 125                                # up to 2^127
    x[1::4, :, ::7] *= 2.0 ** 60                        # squares past fp32 beside small numbers
    w = (1 + torch.rand(n, generator=torch.Generator().manual_seed(n)) * 60).to(TORCH[dtype]).cuda()
    norm = binding.RMSNorm(n, eps=1e-5)
    want, _ = plain(x, w, None, 1e-5, 0.0)
    near(norm.apply(x, w), want, "y")
    near(norm.apply(x, w, residual=torch.zeros_like(x))[0], want, "with a residual")
    given = torch.full((1,), 0.5, device="cuda")
    for scaling, group in (("row", 0), ("group", 32), ("group", 128), ("tensor", 0)):
        codes, scales, _ = norm.quantise(x, w, scaling=scaling, group=group or 128, scales=given if scaling == "tensor" else None)
        size = n if scaling != "group" else group
        parts = -(-n // size)
        padded = torch.nn.functional.pad(want, (0, parts * size - n)).unflatten(-1, (parts, size))
        most = padded.abs().amax(-1) / 448
        if scaling != "tensor":
            assert ((scales.view(most.shape).double() - most).abs() <= most * (Y_ERR + 2.0 ** -23)).all(), (scaling, group)
        each = (scales if scaling == "tensor" else scales.view(most.shape)[..., None].expand(-1, -1, -1, size).flatten(-2)[..., :n])
        check_codes(codes, each.expand(want.shape), want, (scaling, group))


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("eps", [0.0, 1e-44, 1e-36])
@pytest.mark.parametrize("rows,heads,n", FAR)
def test_rows_whose_squares_vanish(dtype, eps, rows, heads, n):
    """Under an eps that does not cover them, rows of small numbers are normed as others are."""
    x = _make(rows, heads, n, dtype)
    for i, e in enumerate((0, -60, -76, -100, -126, -135 if dtype == "f32" else -130)):      # (the last ones subnormal)
        x[i::6] *= 2.0 ** e
    x[:, :, ::5] *= 2.0 ** -20                          # smaller numbers beside larger ones
    w = (0.5 + torch.rand(n, generator=torch.Generator().manual_seed(n))).to(TORCH[dtype]).cuda()
    norm = binding.RMSNorm(n, eps=eps)
    want, _ = plain(x, w, None, float(torch.tensor(eps)), 0.0)
    y = norm.apply(x, w)
    near(y, want, "y")
    near(norm.apply(x, w, residual=torch.zeros_like(x))[0], want, "with a residual")
    for scaling, group in (("row", 0), ("group", 64)):
        codes, scales, _ = norm.quantise(x, w, scaling=scaling, group=group or 128)
        size = group or n
        parts = -(-n // size)
        padded = torch.nn.functional.pad(want, (0, parts * size - n)).unflatten(-1, (parts, size))
        most = (padded.abs().amax(-1) / 448).clamp(min=2.0 ** -126)
        off = most * (Y_ERR + 2.0 ** -23) + 2.0 ** -149
        assert ((scales.view(most.shape).double() - most).abs() <= off).all(), (scaling, group)
        each = scales.view(most.shape)[..., None].expand(-1, -1, -1, size).flatten(-2)[..., :n]
        check_codes(codes, each, want, (scaling, group))
    # a row of zeros has no direction: NaN without eps, as with every other size
    x[0] = 0
    assert norm.apply(x, w)[0].isnan().all() == (float(torch.tensor(eps)) == 0)
