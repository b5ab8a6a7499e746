"""Rotary positions, the quantising write of rows into a cache, and the read back: refusals and
frequencies on the CPU, results on the GPU against plain float64 forms."""
import ctypes
import math
import os
import shutil
import subprocess
from fractions import Fraction

import pytest
import torch

from _rows import (Layout, TORCH, frequencies, half_step, rotate, rotate_bound)
from decode_attention_attn_gb300 import binding, build as lib_build

A = 0x100000   # an aligned address that no refused call dereferences


@pytest.fixture(scope="module", autouse=True)
def built():
    lib_build.build()


# ---- CPU: frequencies and refusals ----------------------------------------------------------
@pytest.mark.parametrize("kw", [
    dict(rotary=128), dict(rotary=64, base=500000.0), dict(rotary=2),
    dict(rotary=128, scaling="linear", factor=4.0),
    dict(rotary=96, scaling="ntk", factor=8.0), dict(rotary=2, scaling="ntk", factor=8.0),
    dict(rotary=128, base=500000.0, scaling="by_parts", factor=8.0, original=8192, low=1.0, high=4.0),
    dict(rotary=128, scaling="by_parts", factor=16.0, original=4096, low=1.0, high=32.0),
    dict(rotary=128, scaling="by_index", factor=16.0, original=4096, low=1.0, high=32.0),
    dict(rotary=64, scaling="by_index", factor=0.5, original=100, low=0.001, high=5000.0),
])
def test_frequencies(kw):
    r = binding.Rope(128, rotary_dim=kw["rotary"], base=kw.get("base", 10000.0),
                     scaling=kw.get("scaling", "none"), factor=kw.get("factor", 1.0),
                     original_max_position=kw.get("original", 0.0), low=kw.get("low", 1.0),
                     high=kw.get("high", 32.0))
    got = torch.tensor(r.frequencies(), dtype=torch.float64)
    # pow and log of two libraries: a few ulps
    assert torch.allclose(got, frequencies(**kw), rtol=1e-13, atol=0)


@pytest.mark.parametrize("kw,code", [
    (dict(head_dim=0), -2), (dict(head_dim=258), -2), (dict(head_dim=127), -2),
    (dict(rotary_dim=0), -2), (dict(rotary_dim=130), -2), (dict(rotary_dim=63), -2),
    (dict(base=1.0), -1), (dict(base=math.inf), -1), (dict(base=math.nan), -1),
    (dict(attn_factor=math.nan), -1), (dict(attn_factor=1e300), -1), (dict(scaling="linear", factor=0.0), -1),
    (dict(scaling="ntk", factor=-2.0), -1), (dict(scaling="linear", factor=math.inf), -1),
    (dict(scaling="by_parts", factor=2.0), -1),                     # no original length
    (dict(scaling="by_parts", factor=2.0, original_max_position=64, low=4.0, high=4.0), -1),
    (dict(scaling="by_index", factor=2.0, original_max_position=64, low=0.0), -1),
    (dict(scaling="ntk", factor=1e300, rotary_dim=4), -1),          # the base overflows
])
def test_rope_refuses_bad_configurations(kw, code):
    with pytest.raises(binding.DecodeAttnError) as e:
        binding.Rope(**{"head_dim": 128, **kw})
    assert e.value.code == code


def test_rope_refuses_unknown_scalings_and_layouts():
    with pytest.raises(ValueError):
        binding.Rope(128, scaling="other")
    for bad in (dict(scaling=5), dict(scaling=-1), dict(interleaved=2)):
        cfg = binding.da_rope_config(128, 128, 0, 0, 10000.0, 1.0, 0.0, 1.0, 32.0, 1.0)
        for k, v in bad.items():
            setattr(cfg, k, v)
        with pytest.raises(binding.DecodeAttnError) as e:
            binding.decode_attn_rope_create(cfg)
        assert e.value.code == -1


def _refused(fn, handle, args, **kw):
    for k, v in kw.items():
        assert hasattr(args, k)
        setattr(args, k, v)
    with pytest.raises(binding.DecodeAttnError) as e:
        fn(handle, args)
    return e.value.code


def test_rope_apply_refuses_bad_arguments():
    r = binding.Rope(128)

    def call(**kw):
        args = binding.da_rope_args(A, A + 65536, 2, 4, 8, 1024, 128, 1024, 128, A, 0, None)
        return _refused(binding.decode_attn_rope_apply, r.handle, args, **kw)

    assert call(x=None) == -1 and call(out=None) == -1 and call(positions=None) == -1
    assert call(rows=-1) == -1 and call(heads=0) == -1 and call(transpose=2) == -1
    assert call(dtype=3) == -2 and call(dtype=-1) == -2 and call(heads=(1 << 20) + 1) == -2
    assert call(x=A + 1) == -1 and call(out=A + 3) == -1 and call(positions=A + 2) == -1
    assert call(out=A, out_row_stride=2048) == -1          # in place with other strides
    assert call(out_head_stride=127) == -1 and call(out_head_stride=0) == -1    # rows on one another
    assert call(out_row_stride=1023) == -1 and call(out_row_stride=128) == -1
    assert call(out_row_stride=0) == -1 and call(out_row_stride=-1024) == -1
    # no rows: nothing is enqueued, no pointer is looked at
    args = binding.da_rope_args(None, None, 2, 0, 8, 1024, 128, 1024, 128, None, 0, None)
    binding.decode_attn_rope_apply(r.handle, args)


def _plan(**kw):
    base = dict(batch=4, num_q_heads=32, num_kv_heads=8, head_dim=128, qkv_dtype="bf16",
                out_dtype="bf16", paged=True, page_size=16, max_blocks_per_seq=8,
                num_physical_blocks=64, num_sms=152)
    return binding.decode_attn_plan(binding.make_problem(**{**base, **kw}), 0)


def test_kv_write_refuses_bad_arguments():
    plan, ws = _plan()
    r, short = binding.Rope(128), binding.Rope(64)

    def call(plan=plan, **kw):
        args = binding.da_kv_write_args(A, A, 1024, 128, 1024, 128, 4, A, A, A, A, A, r.handle, A, A,
                                        A + 65536, 4096, 128, 4096, 128, A, A, ws, None)
        return _refused(binding.decode_attn_kv_write, plan, args, **kw)

    for name in ("k", "v", "k_cache", "v_cache", "block_table", "row_offsets", "start"):
        assert call(**{name: None}) == -1, name
    assert call(rows=-1) == -1
    assert call(k=A + 1) == -1 and call(k_cache=A + 8) == -1 and call(start=A + 2) == -1
    assert call(row_offsets=A + 1) == -1 and call(block_table=A + 2) == -1
    assert call(positions=A + 1) == -1 and call(amax=A + 2) == -1 and call(q=A + 1) == -1
    assert call(q=None) == -1 and call(q_out=None) == -1     # one without the other
    assert call(rope=None) == -1                             # q and positions without a rope
    assert call(rope=None, positions=None) == -1
    assert call(rope=short.handle) == -1                     # another head_dim
    assert call(q_out=A, q_out_row_stride=8192) == -1        # in place with other strides
    assert call(q_out_row_stride=4095) == -1 and call(q_out_head_stride=64) == -1
    assert call(workspace=A + 16) == -1 and call(workspace_bytes=ws - 1) == -3
    contiguous, _ = _plan(paged=False, max_seq_len=64)
    assert call(contiguous) == -1                            # a table for a contiguous cache
    checked, _ = _plan(validate=True)
    assert call(checked, workspace=None) == -1               # validate needs the status word
    tiny, _ = _plan(kv_dtype="e4m3", k_scale=1e-45)
    assert call(tiny) == -1                                  # 1 / k_scale is no fp32 number
    for p in (plan, contiguous, checked, tiny):
        binding.decode_attn_destroy(p)


def test_kv_read_refuses_bad_arguments():
    plan, ws = _plan()

    def call(plan=plan, **kw):
        args = binding.da_kv_read_args(A, A, A, A, A, 4, A, A + 65536, A, ws, None)
        return _refused(binding.decode_attn_kv_read, plan, args, **kw)

    for name in ("k_cache", "v_cache", "block_table", "row_offsets", "start", "k_out", "v_out"):
        assert call(**{name: None}) == -1, name
    assert call(k_cache=None, k_out=None, v_cache=None, v_out=None) == -1
    assert call(rows=-1) == -1 and call(k_out=A + 8) == -1 and call(v_cache=A + 4) == -1
    assert call(v_out=A) == -1 and call(v_out=A + 16) == -1       # results on one another
    assert call(workspace=A + 16) == -1 and call(workspace_bytes=ws - 1) == -3
    binding.decode_attn_destroy(plan)


def test_null_handles_are_refused():
    L = binding.lib()
    plan, _ = _plan()
    assert L.decode_attn_rope_create(None, None) == -1
    assert L.decode_attn_rope_frequencies(None, None) == -1
    assert L.decode_attn_rope_apply(None, None) == -1
    assert L.decode_attn_kv_write(plan, None) == -1 and L.decode_attn_kv_read(plan, None) == -1
    L.decode_attn_rope_destroy(None)
    binding.decode_attn_destroy(plan)


def test_wrappers_refuse_bad_tensors():
    lay = Layout([3, 4], [1, 2], 2, 64, page=16)
    io = binding.KVCacheIO(lay.problem)
    kc, vc = lay.cache(), lay.cache()
    k = lay.normal(lay.rows, 2, 64)
    args = [k, k, kc, vc, lay.table, lay.row_offsets, lay.start]
    with pytest.raises(ValueError, match="CUDA"):
        io.write(*args)

    def bad(i, t, **kw):
        with pytest.raises(ValueError):
            io.write(*[t if j == i else x for j, x in enumerate(args)], **kw)

    bad(0, k.float())
    bad(0, k[:, :1])
    bad(1, k[:2])
    bad(2, kc[:1])
    bad(4, None)
    bad(4, lay.table.long())
    bad(5, lay.row_offsets[:-1])
    bad(6, lay.start.float())
    bad(0, k, q=lay.normal(lay.rows, 2, 64))                  # q without a rope
    bad(0, k, q_out=k)
    with pytest.raises(ValueError):
        io.read(kc, vc, lay.table, lay.row_offsets, lay.start, None, None)
    with pytest.raises(ValueError):
        io.read(None, vc, lay.table, lay.row_offsets, lay.start, k, k)
    with pytest.raises(ValueError):
        io.check_status()
    r = binding.Rope(64)
    with pytest.raises(ValueError):
        r.apply(k.double(), lay.start)
    with pytest.raises(ValueError):
        r.apply(k, torch.zeros(lay.rows, dtype=torch.int32))  # not on a GPU


# ---- GPU: rotary ------------------------------------------------------------------------------
def _check_rotated(got, x, pos, theta, rotary, interleaved, m, transpose=False):
    ref = rotate(x.double(), pos, theta, rotary, interleaved, m, transpose)
    tol = rotate_bound(x.double(), pos, theta, rotary, interleaved, m)
    tol[..., :rotary] += ref[..., :rotary].abs() * half_step(x.dtype) * 1.001 + 6e-8
    assert ((got.cpu().double() - ref).abs() <= tol).all()


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("d,rotary", [(128, 128), (128, 32), (64, 64), (64, 2), (256, 256), (66, 34), (2, 2)])
def test_rope(dtype, interleaved, d, rotary):
    g = torch.Generator().manual_seed(d + rotary)
    pos = torch.tensor([0, 1, -1, 7, 1000003, 2 ** 31 - 1, -2 ** 31, 131071, 4095], dtype=torch.int32)
    x = torch.randn(len(pos), 5, d, generator=g).to(TORCH[dtype])
    r = binding.Rope(d, rotary, interleaved, base=500000.0, scaling="by_parts", factor=8.0,
                     original_max_position=8192, low=1.0, high=4.0, attn_factor=1.25)
    theta = torch.tensor(r.frequencies(), dtype=torch.float64)
    for transpose in (False, True):
        got = r.apply(x.cuda(), pos.cuda(), transpose=transpose)
        _check_rotated(got, x, pos, theta, rotary, interleaved, 1.25, transpose)
        assert torch.equal(got.cpu()[..., rotary:], x[..., rotary:])


@pytest.mark.gpu
@pytest.mark.parametrize("offset,gap", [(0, 3), (1, 0), (8, 1), (3, 2)])
@pytest.mark.parametrize("rows", [1, 700])
def test_rope_strided_unaligned_and_in_place(offset, gap, rows):
    d, heads = 64, 6
    g = torch.Generator().manual_seed(offset)
    base = torch.randn(offset + rows * (heads + gap) * d + 8, generator=g).bfloat16()
    pos = torch.randint(0, 5000, (rows,), generator=g, dtype=torch.int32)
    r = binding.Rope(d)
    theta = torch.tensor(r.frequencies(), dtype=torch.float64)
    view = lambda t: t[offset:offset + rows * (heads + gap) * d].view(rows, heads + gap, d)[:, :heads]
    dev = base.cuda()
    got = r.apply(view(dev), pos.cuda())
    _check_rotated(got, view(base), pos, theta, d, False, 1.0)
    same = r.apply(view(dev), pos.cuda(), out=view(dev))
    assert same.data_ptr() == view(dev).data_ptr() and torch.equal(same, got)
    back = dev.cpu()
    view(back).copy_(view(base))          # nothing but the rotated heads changed
    assert torch.equal(back, base)


@pytest.mark.gpu
def test_rope_broadcast_rows_and_heads_first():
    """One row read for all positions, and a [heads, rows, d] output."""
    d = 128
    pos = torch.arange(50, dtype=torch.int32)
    x = torch.randn(1, 3, d, generator=torch.Generator().manual_seed(0)).half()
    r = binding.Rope(d)
    theta = torch.tensor(r.frequencies(), dtype=torch.float64)
    out = torch.zeros(3, 50, d, dtype=torch.float16, device="cuda").transpose(0, 1)
    got = r.apply(x.cuda().expand(50, 3, d), pos.cuda(), out=out)
    assert got.stride() == (d, 50 * d, 1)
    _check_rotated(got, x.expand(50, 3, d), pos, theta, d, False, 1.0)


@pytest.mark.gpu
@pytest.mark.parametrize("interleaved", [False, True])
def test_rope_gradient(interleaved):
    """transpose=True against autograd of the formula and against differences of the forward call."""
    rows, heads, d, rotary = 33, 3, 64, 32
    g = torch.Generator().manual_seed(1)
    x, dy, dx = (torch.randn(rows, heads, d, generator=g) for _ in range(3))
    pos = torch.randint(0, 9000, (rows,), generator=g, dtype=torch.int32)
    r = binding.Rope(d, rotary, interleaved, attn_factor=0.75)
    theta = torch.tensor(r.frequencies(), dtype=torch.float64)
    leaf = x.double().requires_grad_()
    rotate(leaf, pos, theta, rotary, interleaved, 0.75).backward(dy.double())
    grad = r.apply(dy.cuda(), pos.cuda(), transpose=True).cpu()
    tol = rotate_bound(dy.double(), pos, theta, rotary, interleaved, 0.75) + leaf.grad.abs() * 2.0 ** -23
    assert ((grad.double() - leaf.grad).abs() <= tol).all()
    # <dy, R(x + dx) - R(x)> = <R^T dy, dx>: the map is linear, so the difference is exact but for
    # roundings (2^-21 of the sums of magnitudes bounds the forward errors of both calls)
    moved = r.apply((x + dx).cuda(), pos.cuda()).cpu().double() - r.apply(x.cuda(), pos.cuda()).cpu().double()
    step = (x + dx).double() - x.double()
    left, right = (dy.double() * moved).sum(), (grad.double() * step).sum()
    size = (dy.double().abs().sum(-1) * (x.abs() + (x + dx).abs()).double().amax(-1)).sum()
    assert abs(left - right) <= size * 2.0 ** -19


@pytest.mark.gpu
def test_rope_without_rows():
    r = binding.Rope(64)
    x = torch.empty(0, 4, 64, device="cuda")
    assert r.apply(x, torch.empty(0, dtype=torch.int32, device="cuda")).shape == (0, 4, 64)


# ---- GPU: writes ------------------------------------------------------------------------------
LAYOUTS = {
    "decode": dict(held=[5, 0, 130, 77], new=[1, 1, 1, 1]),
    "ragged": dict(held=[0, 31, 500, 7, 16], new=[40, 0, 3, 129, 0]),
    "padded": dict(held=[9, 2], new=[3, 14], before=5, behind=6),
    "one": dict(held=[0], new=[1]),
}
KINDS = [("f32", "f32"), ("f16", "f16"), ("bf16", "bf16"), ("bf16", "e4m3")]


def _expected_write(lay, cache, rows, z_of, scale):
    """(float64 values of the flat cache after the write, which rows of it were written)."""
    ref = lay.values(cache, scale).clone()
    hit = torch.zeros(ref.shape[0], dtype=torch.bool)
    for r, z in z_of:
        ref[z], hit[z] = rows[r], True
    return ref, hit


def _check_cache(lay, after, before, ref, hit, scale, slack):
    """Rows not written keep their bits; written ones are the nearest stored values."""
    flat_a, flat_b = (c.cpu().reshape(-1, lay.hkv, lay.d) for c in (after, before))
    assert torch.equal(flat_a[~hit].view(torch.uint8), flat_b[~hit].view(torch.uint8))
    got = lay.values(after.cpu(), scale)[hit]
    want = ref[hit]
    if lay.kv == "e4m3":
        want = want.clamp(-448 * scale, 448 * scale)
        # half a step: 2^-4 of a normal value, 2^-10 below the smallest normal; 1 / scale is off by 2^-24
        # and its product by 2^-24
        tol = torch.maximum(want.abs() * 2.0 ** -4, torch.tensor(2.0 ** -10 * scale, dtype=torch.float64))
        tol = tol * (1 + 2.0 ** -20)
    else:
        tol = want.abs() * half_step(TORCH[lay.dtype]) + (2.0 ** -25 if lay.dtype == "f16" else 0)
    assert ((got - want).abs() <= tol + slack[hit]).all()


@pytest.mark.gpu
@pytest.mark.parametrize("dtype,kv", KINDS)
@pytest.mark.parametrize("name", list(LAYOUTS))
@pytest.mark.parametrize("page,hkv,d", [(0, 2, 64), (16, 8, 128), (8, 3, 64), (256, 1, 128)])
@pytest.mark.parametrize("rope", [None, "half", "part"])
def test_kv_write(dtype, kv, name, page, hkv, d, rope):
    lay = Layout(**LAYOUTS[name], hkv=hkv, d=d, page=page, hq=4 * hkv, dtype=dtype, kv=kv, seed=3)
    io = binding.KVCacheIO(lay.problem, findings=True)
    kc, vc = lay.cache(), lay.cache()
    wide = lay.normal(lay.rows, 6 * hkv, d)
    q, k, v = wide[:, :4 * hkv], wide[:, 4 * hkv:5 * hkv], wide[:, 5 * hkv:]
    z_of = [(r, lay.cache_row(b, t)) for r, (b, t) in enumerate(zip(lay.row_seq, lay.row_pos)) if b >= 0]
    dev = wide.cuda()
    dq, dk, dv = dev[:, :4 * hkv], dev[:, 4 * hkv:5 * hkv], dev[:, 5 * hkv:]
    gk, gv = kc.cuda(), vc.cuda()
    place = (lay.table.cuda() if page else None, lay.row_offsets.cuda(), lay.start.cuda())
    k_ref, k_slack = k.double(), torch.zeros(lay.rows, hkv, d, dtype=torch.float64)
    if rope:
        rd, inter = (d, False) if rope == "half" else (d // 2, True)
        R = binding.Rope(d, rd, inter)
        theta = torch.tensor(R.frequencies(), dtype=torch.float64)
        pos = torch.tensor(lay.row_pos, dtype=torch.int32)
        other = None
        if rope == "part":               # positions of their own
            pos = torch.randint(0, 100000, (lay.rows,), generator=lay.gen, dtype=torch.int32)
            other = pos.cuda()
        out = torch.full((lay.rows, 4 * hkv, d), 7.0, dtype=TORCH[dtype], device="cuda")
        io.write(dk, dv, gk, gv, *place, rope=R, positions=other, q=dq, q_out=out)
        member = torch.tensor([b >= 0 for b in lay.row_seq])
        _check_rotated(out[member.cuda()], q[member], pos[member], theta, rd, inter, 1.0)
        assert (out[~member.cuda()] == 7.0).all()
        k_ref = rotate(k.double(), pos, theta, rd, inter)
        k_slack = rotate_bound(k.double(), pos, theta, rd, inter)
    else:
        assert io.write(dk, dv, gk, gv, *place) is None
    io.check_status()
    flat = torch.zeros(lay.values(kc, 1.0).shape, dtype=torch.float64)
    slack_k = flat.clone()
    for r, z in z_of:
        slack_k[z] = k_slack[r] * 1.07      # rounding moves with the value: 1 + 2^-4
    _check_cache(lay, gk, kc, *_expected_write(lay, kc, k_ref, z_of, lay.k_scale), lay.k_scale, slack_k)
    _check_cache(lay, gv, vc, *_expected_write(lay, vc, v.double(), z_of, lay.v_scale), lay.v_scale, flat)


@pytest.mark.gpu
def test_kv_write_unaligned_rows_equal_aligned_ones():
    """Rows at odd element offsets and strides take the one-pair-a-lane kernel: same bits."""
    for dtype, kv in KINDS:
        lay = Layout([3, 40], [5, 2], 2, 64, page=16, hq=4, dtype=dtype, kv=kv)
        io = binding.KVCacheIO(lay.problem)
        R = binding.Rope(64, 32, True)
        n = lay.rows * 8 * 64
        base = lay.normal(n + 1).cuda()
        place = (lay.table.cuda(), lay.row_offsets.cuda(), lay.start.cuda())
        got = []
        for rows in (base[1:].view(lay.rows, 8, 64), base[1:].view(lay.rows, 8, 64).clone()):
            kc, vc = (torch.zeros(lay.shape, dtype=torch.uint8 if kv == "e4m3" else TORCH[dtype], device="cuda")
                      for _ in range(2))
            q = io.write(rows[:, 4:6], rows[:, 6:], kc, vc, *place, rope=R, q=rows[:, :4])
            got.append((kc, vc, q))
        assert all(torch.equal(a, b) for a, b in zip(*got))


@pytest.mark.gpu
def test_kv_write_corner_values_to_fp8():
    """Ties to even, saturation, infinities, NaN, zeros and subnormals, all 256 codes included."""
    lay = Layout([0], [2], 1, 128, kv="e4m3", k_scale=0.25, v_scale=2.0)
    codes = torch.arange(256, dtype=torch.uint8).view(2, 1, 128)
    exact = codes.view(torch.float8_e4m3fn).float()
    grid = torch.sort(torch.cat([exact.flatten()[torch.isfinite(exact.flatten())].unique()]))[0]
    ties = (grid[1:] + grid[:-1]) / 2
    special = torch.tensor([460.0, 464.0, 465.0, 1e30, -1e30, math.inf, -math.inf, math.nan, 0.0, -0.0])
    rows = torch.cat([ties, special])[:256]
    rows = torch.cat([rows, torch.zeros(256 - len(rows))]).view(2, 1, 128)
    for values in (exact, rows):
        k, v = (values * 0.25).bfloat16(), (values * 2.0).bfloat16()
        io = binding.KVCacheIO(lay.problem)
        kc, vc = (torch.zeros(lay.shape, dtype=torch.uint8, device="cuda") for _ in range(2))
        io.write(k.cuda(), v.cuda(), kc, vc, None, lay.row_offsets.cuda(), lay.start.cuda())
        for x, c, inv in ((k, kc, 4.0), (v, vc, 0.5)):
            want = (x.float() * inv).clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)
            got = c.cpu().view(2, 1, 128)
            nan = torch.isnan(x.float())
            assert torch.equal(got[~nan], want[~nan])
            assert ((got[nan] & 0x7F) == 0x7F).all()


@pytest.mark.gpu
@pytest.mark.parametrize("dtype,kv", [("bf16", "e4m3"), ("f16", "f16")])
@pytest.mark.parametrize("rope", [False, True])
def test_kv_write_amax(dtype, kv, rope):
    lay = Layout([3, 4, 0], [7, 0, 300], 2, 64, page=8, dtype=dtype, kv=kv, before=3, behind=3)
    io = binding.KVCacheIO(lay.problem)
    k, v = lay.normal(lay.rows, 2, 64), lay.normal(lay.rows, 2, 64)
    k[0], v[-1] = 1000.0, 1000.0          # rows of no sequence do not count
    k[5, 0, 3] = math.nan
    R = binding.Rope(64) if rope else None
    kc, vc = lay.cache().cuda(), lay.cache().cuda()
    amax = torch.zeros(2, device="cuda")
    place = (lay.table.cuda(), lay.row_offsets.cuda(), lay.start.cuda())
    io.write(k.cuda(), v.cuda(), kc, vc, *place, rope=R, amax=amax)
    member = torch.tensor([b >= 0 for b in lay.row_seq])
    pos = torch.tensor(lay.row_pos, dtype=torch.int32)
    kr = rotate(k.double(), pos, torch.tensor(R.frequencies(), dtype=torch.float64), 64) if rope else k.double()
    want = [kr[member].nan_to_num(0.0).abs().max().item(), v[member].double().abs().max().item()]
    assert amax.cpu().double().tolist() == pytest.approx(want, rel=2e-6)
    first = amax.clone()
    io.write((k * 0.5).cuda(), (v * 2).cuda(), kc, vc, *place, rope=R, amax=amax)    # a running maximum
    assert amax[0] == first[0] and amax[1] == 2 * first[1]


@pytest.mark.gpu
@pytest.mark.parametrize("page", [0, 16])
def test_rows_without_a_place_are_recorded_and_not_written(page):
    lay = Layout([30, 3, 2], [2, 2, 2], 2, 64, page=page, capacity=32, kv="e4m3")
    io = binding.KVCacheIO(lay.problem, findings=True)
    kc, vc = lay.cache().cuda(), lay.cache().cuda()
    k = lay.normal(lay.rows, 2, 64).cuda()
    table = lay.table.cuda() if page else None
    place = lambda start: (table, lay.row_offsets.cuda(), torch.tensor(start, dtype=torch.int32, device="cuda"))

    def code():
        try:
            io.check_status()
        except binding.DecodeAttnError as e:
            return e.code
        return 0

    before = kc.clone()
    io.write(k, k, kc, vc, *place([31, -1, 32]))          # rows at 31 and 0 have a place, the others not
    assert code() == -7 and code() == 0
    changed = (kc != before).view(-1, 2, 64).any(-1).any(-1)
    assert changed.sum() == 2 and changed[lay.cache_row(0, 31)] and changed[lay.cache_row(1, 0)]
    out_k, out_v = (torch.full((lay.rows, 2, 64), 3.0, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    io.read(kc, vc, *place([31, -1, 2147483647]), out_k, out_v)
    assert code() == -7
    assert (out_k[1] == 0).all() and (out_v[2] == 0).all() and (out_k[4:] == 0).all()
    assert (out_k[0] != 0).any() and (out_k[3] != 0).any()
    if page:
        for entry in (-1, lay.pool, 2 ** 31 - 1):
            table[1, 0] = entry
            before = kc.clone()
            io.write(k, k, kc, vc, *place([0, 3, 2]))
            assert code() == -4
            changed = (kc != before).view(-1, 2, 64).any(-1).any(-1)
            assert changed.sum() <= 4
            io.read(kc, vc, *place([0, 3, 2]), out_k, out_v)
            assert code() == -4 and (out_k[2:4] == 0).all() and (out_v[2:4] == 0).all()
    strict = Layout([30, 3, 2], [2, 2, 2], 2, 64, page=page, capacity=32, kv="e4m3", validate=True)
    io = binding.KVCacheIO(strict.problem)
    with pytest.raises(binding.DecodeAttnError) as e:
        io.write(k, k, kc, vc, strict.table.cuda() if page else None, *place([31, 3, 2])[1:])
    assert e.value.code == -7
    io.write(k, k, kc, vc, strict.table.cuda() if page else None, *place([30, 3, 2])[1:])


# ---- GPU: reads -------------------------------------------------------------------------------
@pytest.mark.gpu
@pytest.mark.parametrize("dtype,kv", KINDS)
@pytest.mark.parametrize("name", list(LAYOUTS))
@pytest.mark.parametrize("page,hkv,d", [(0, 2, 64), (16, 8, 128), (8, 3, 64), (256, 1, 64), (16, 1, 128)])
def test_kv_read(dtype, kv, name, page, hkv, d):
    lay = Layout(**LAYOUTS[name], hkv=hkv, d=d, page=page, dtype=dtype, kv=kv, seed=5)
    io = binding.KVCacheIO(lay.problem)
    caches = [lay.cache(), lay.cache()]
    place = (lay.table.cuda() if page else None, lay.row_offsets.cuda(), lay.start.cuda())
    for which in ((0, 1), (0,), (1,)):
        src = [caches[i].cuda() if i in which else None for i in range(2)]
        out = [torch.full((lay.rows, hkv, d), 9.0, dtype=TORCH[dtype], device="cuda") if i in which else None
               for i in range(2)]
        io.read(*src, *place, *out)
        for i, scale in zip(range(2), (lay.k_scale, lay.v_scale)):
            if out[i] is None:
                continue
            want = torch.full((lay.rows, hkv, d), 9.0, dtype=TORCH[dtype])
            flat = caches[i].reshape(-1, hkv, d)
            for r, (b, t) in enumerate(zip(lay.row_seq, lay.row_pos)):
                if b >= 0:
                    row = flat[lay.cache_row(b, t)]
                    if kv == "e4m3":   # one fp32 product, one rounding
                        row = (row.view(torch.float8_e4m3fn).float() * torch.tensor(scale)).to(TORCH[dtype])
                    want[r] = row
            assert torch.equal(out[i].cpu(), want)


@pytest.mark.gpu
@pytest.mark.parametrize("scale", [0.0125, 1.0, 3.7e-5, 911.0])
def test_rows_read_from_fp8_and_written_back_keep_their_codes(scale):
    lay = Layout([0, 0], [100, 37], 2, 128, page=16, kv="e4m3", k_scale=scale, v_scale=scale)
    io = binding.KVCacheIO(lay.problem)
    kc = lay.cache().cuda()
    place = (lay.table.cuda(), lay.row_offsets.cuda(), lay.start.cuda())
    k, v = (torch.empty(lay.rows, 2, 128, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    io.read(kc, kc, *place, k, v)
    back = kc.clone()
    io.write(k, v, back, torch.zeros_like(kc), *place)
    assert torch.equal(back, kc)


@pytest.mark.gpu
def test_offsets_past_32_bits():
    """A pool of more than 2^31 elements: rows at its far end."""
    page, hkv, d = 256, 8, 128
    pool = 2 ** 31 // (page * hkv * d) + 9
    prob = binding.make_problem(batch=2, num_q_heads=8, num_kv_heads=hkv, head_dim=d, qkv_dtype="bf16",
                                out_dtype="bf16", paged=True, page_size=page, max_blocks_per_seq=2,
                                num_physical_blocks=pool, kv_dtype="e4m3", k_scale=0.5, v_scale=0.5)
    io = binding.KVCacheIO(prob)
    kc, vc = (torch.zeros((pool, page, hkv, d), dtype=torch.uint8, device="cuda") for _ in range(2))
    table = torch.tensor([[pool - 1, pool - 2], [0, pool - 3]], dtype=torch.int32, device="cuda")
    offs = torch.tensor([0, 3, 300], dtype=torch.int32, device="cuda")
    start = torch.tensor([254, 100], dtype=torch.int32, device="cuda")
    k = torch.randint(-8, 8, (300, hkv, d), device="cuda").bfloat16()
    io.write(k, -k, kc, vc, table, offs, start)
    a, b = torch.empty_like(k), torch.empty_like(k)
    io.read(kc, vc, table, offs, start, a, b)
    assert torch.equal(a, k) and torch.equal(b, -k)
    assert torch.equal(kc[pool - 1, 255].view(torch.float8_e4m3fn).float() * 0.5, k[1].float())


# ---- GPU: streams and graphs ------------------------------------------------------------------
@pytest.mark.gpu
def test_captured_write_and_read_follow_their_inputs():
    lay = Layout([3, 9], [4, 2], 2, 64, page=16, hq=4, kv="e4m3", capacity=64)
    io = binding.KVCacheIO(lay.problem)
    R = binding.Rope(64)
    kc, vc = lay.cache().cuda(), lay.cache().cuda()
    table, offs, start = lay.table.cuda(), lay.row_offsets.cuda(), lay.start.cuda()
    rows = lay.normal(lay.rows, 8, 64).cuda()
    q_out = torch.empty(lay.rows, 4, 64, dtype=torch.bfloat16, device="cuda")
    k_out, v_out = (torch.empty(lay.rows, 2, 64, dtype=torch.bfloat16, device="cuda") for _ in range(2))

    def step(out, ko, vo, kc, vc):
        io.write(rows[:, 4:6], rows[:, 6:], kc, vc, table, offs, start, rope=R, q=rows[:, :4], q_out=out)
        io.read(kc, vc, table, offs, start, ko, vo)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step(q_out, k_out, v_out, kc, vc)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step(q_out, k_out, v_out, kc, vc)
    for n in range(2):
        rows.copy_(lay.normal(lay.rows, 8, 64))
        start.copy_(torch.tensor([5 + n, 1], dtype=torch.int32))
        ref_kc, ref_vc, ref = kc.clone(), vc.clone(), [torch.empty_like(t) for t in (q_out, k_out, v_out)]
        step(*ref, ref_kc, ref_vc)
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip((q_out, k_out, v_out, kc, vc), (*ref, ref_kc, ref_vc)):
            assert torch.equal(a, b)


@pytest.mark.gpu
@pytest.mark.parametrize("k_scale,v_scale", [(0.01171875, 0.0087890625), (0.0125, 0.0075), (3.1, 1e-20), (7e20, 1 / 3), (0.25, 2e38)])
@pytest.mark.parametrize("aligned", [True, False])
def test_codes_are_those_of_the_fp32_quotient(k_scale, v_scale, aligned):
    """Every bf16 value of +-480 scales and less: the codes of x / scale in fp32, next to ties between two codes
    too, where a product with the rounded reciprocal falls to the other side."""
    x = torch.arange(65536, dtype=torch.int32).to(torch.int16).view(torch.bfloat16).float()
    x = x[torch.isfinite(x)]
    lay = Layout([0], [len(x) // 128], 1, 128, kv="e4m3", k_scale=k_scale, v_scale=v_scale)
    x = x[:lay.rows * 128].view(lay.rows, 1, 128)
    x = x.bfloat16()
    rows = torch.zeros(lay.rows * 129 + 1, dtype=torch.bfloat16, device="cuda")
    k = (x.cuda() if aligned else rows[1:].view(lay.rows, 1, 129)[:, :, :128].copy_(x))
    kc, vc = (torch.zeros(lay.shape, dtype=torch.uint8, device="cuda") for _ in range(2))
    binding.KVCacheIO(lay.problem).write(k, k, kc, vc, None, lay.row_offsets.cuda(), lay.start.cuda())
    for c, scale in ((kc, k_scale), (vc, v_scale)):
        want = (x.float() / torch.tensor(scale)).clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)
        assert torch.equal(c.cpu().view(want.shape), want)


# ---- results over inputs ----------------------------------------------------------------------
def test_where_rows_lie(tmp_path):
    cxx = shutil.which("g++") or shutil.which("c++")
    if cxx is None:
        pytest.skip("no host C++ compiler")
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    exe = tmp_path / "row_rules"
    subprocess.run([cxx, "-std=c++17", "-O1", "-Wall", "-Werror",
                    "-I" + os.path.join(root, "decode_attention_attn_gb300", "csrc"),
                    os.path.join(root, "tests", "c_row_rules.cpp"), "-o", str(exe)], check=True)
    r = subprocess.run([str(exe)], capture_output=True, text=True)
    assert r.returncode == 0 and r.stdout.strip() == "ok", r.stdout + r.stderr


def test_rope_apply_refuses_results_over_inputs():
    r = binding.Rope(128)

    def call(**kw):   # 8 rows of 4 heads, bf16: rows of 1024 bytes, heads of 256
        args = binding.da_rope_args(A, A + 65536, 2, 8, 4, 512, 128, 512, 128, A, 0, None)
        return _refused(binding.decode_attn_rope_apply, r.handle, args, **kw)

    assert call(out=A + 1024) == -1 and call(out=A - 1024) == -1       # a row on, a row back
    assert call(out=A + 256) == -1 and call(out=A + 2) == -1           # a head on, an element on
    assert call(out=A + 7 * 1024) == -1 and call(x=A + 7 * 1024, out=A) == -1
    assert call(out=A + 4096, out_row_stride=1024) == -1               # other strides of one memory
    assert call(x_row_stride=0, x=A + 65536 + 3 * 1024) == -1          # one row for all, among the results
    assert call(out_row_stride=2 ** 62, out_head_stride=2 ** 61) == -1


def test_kv_write_refuses_results_over_inputs():
    plan, ws = _plan()
    r = binding.Rope(128)
    far = 1 << 24

    def call(**kw):
        args = binding.da_kv_write_args(A, A + far, 1024, 128, 1024, 128, 4, A + 2 * far, A + 3 * far, A, A, A,
                                        r.handle, None, A + 4 * far, A + 5 * far, 4096, 128, 4096, 128, None, None,
                                        0, None)
        return _refused(binding.decode_attn_kv_write, plan, args, **kw)

    assert call(q_out=A + 4 * far + 8192) == -1                        # q, a row on
    assert call(q_out=A + 2048) == -1 and call(q_out=A + far - 16384) == -1   # over k, over v
    assert call(v_cache=A + 2 * far) == -1 and call(v_cache=A + 2 * far + 4096) == -1
    binding.decode_attn_destroy(plan)


@pytest.mark.gpu
def test_parts_of_one_tensor_are_rotated_beside_one_another():
    """Results in other heads, every other head, or other rows of the input's own tensor."""
    d = 64
    base = torch.randn(40, 12, d, generator=torch.Generator().manual_seed(2)).bfloat16()
    pos = torch.arange(40, dtype=torch.int32)
    r = binding.Rope(d)
    theta = torch.tensor(r.frequencies(), dtype=torch.float64)
    for x, out in ((lambda t: t[:, :5], lambda t: t[:, 7:]), (lambda t: t[:, ::2], lambda t: t[:, 1::2]),
                   (lambda t: t[:20], lambda t: t[20:]), (lambda t: t[::2], lambda t: t[1::2]),
                   (lambda t: t.transpose(0, 1)[:, :7], lambda t: t.transpose(0, 1)[:, 9:16])):
        dev = base.cuda()
        p = pos[:x(base).shape[0]]
        r.apply(x(dev), p.cuda(), out=out(dev))
        _check_rotated(out(dev), x(base), p, theta, d, False, 1.0)
        want = base.clone()
        out(want).copy_(out(dev).cpu())
        assert torch.equal(dev.cpu(), want)
        with pytest.raises(binding.DecodeAttnError):
            r.apply(dev[1:], pos[1:].cuda(), out=dev[:-1])


# ---- gradients --------------------------------------------------------------------------------
def test_rope_apply_refuses_an_out_that_autograd_would_lose():
    r = binding.Rope(64)
    x, pos = torch.zeros(3, 2, 64, requires_grad=True), torch.zeros(3, dtype=torch.int32)
    with pytest.raises(ValueError, match="autograd"):
        r.apply(x, pos, out=torch.zeros(3, 2, 64))
    with pytest.raises(ValueError, match="autograd"):
        r.apply(x.detach(), pos, out=x)
    with torch.no_grad(), pytest.raises(ValueError, match="CUDA"):     # not recorded, so not refused for it
        r.apply(x, pos, out=torch.zeros(3, 2, 64))


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("transpose", [False, True])
def test_autograd_records_a_rotation(dtype, interleaved, transpose):
    """backward() through apply: the transposed map of the output's gradient, for a leaf, a strided part of one, a
    row broadcast to all, and an expanded gradient; and through the backward pass itself."""
    rows, heads, d, rotary = 21, 3, 64, 32
    g = torch.Generator().manual_seed(5)
    r = binding.Rope(d, rotary, interleaved, attn_factor=0.75)
    theta = torch.tensor(r.frequencies(), dtype=torch.float64)
    pos = torch.randint(0, 9000, (rows,), generator=g, dtype=torch.int32)
    dy = torch.randn(rows, heads, d, generator=g).to(TORCH[dtype])

    x = torch.randn(rows, 2 * heads, d, generator=g).to(TORCH[dtype]).cuda().requires_grad_()
    y = r.apply(x[:, heads:], pos.cuda(), transpose=transpose)
    assert y.requires_grad and torch.equal(y, r.apply(x.detach()[:, heads:], pos.cuda(), transpose=transpose))
    y.backward(dy.cuda())
    want = rotate(dy.double(), pos, theta, rotary, interleaved, 0.75, not transpose)
    err = rotate_bound(dy.double(), pos, theta, rotary, interleaved, 0.75)
    got = x.grad.cpu().double()
    assert (got[:, :heads] == 0).all()
    assert ((got[:, heads:] - want).abs() <= err + want.abs() * half_step(TORCH[dtype]) * 1.001 + 6e-8).all()
    # one row for all positions: its gradient is the sum of theirs
    one = torch.randn(1, heads, d, generator=g).to(TORCH[dtype]).cuda().requires_grad_()
    r.apply(one.expand(rows, heads, d), pos.cuda(), transpose=transpose).backward(dy.cuda())
    each = want.abs() * half_step(TORCH[dtype]) * 1.001 + err + 6e-8
    total = want.sum(0, keepdim=True)
    tol = each.sum(0, keepdim=True) + want.abs().sum(0, keepdim=True) * 21 * 2.0 ** -23 + \
        total.abs() * half_step(TORCH[dtype]) * 1.001 + 6e-8
    assert ((one.grad.cpu().double() - total).abs() <= tol * 1.01).all()
    # a gradient with no strides, and a gradient of a gradient
    leaf = torch.randn(rows, heads, d, generator=g).to(TORCH[dtype]).cuda().requires_grad_()
    r.apply(leaf, pos.cuda(), transpose=transpose).sum().backward()
    ones = torch.ones(rows, heads, d, dtype=torch.float64)
    want = rotate(ones, pos, theta, rotary, interleaved, 0.75, not transpose)
    err = rotate_bound(ones, pos, theta, rotary, interleaved, 0.75)
    assert ((leaf.grad.cpu().double() - want).abs() <= err + want.abs() * half_step(TORCH[dtype]) * 1.001 + 6e-8).all()
    w = dy.cuda().requires_grad_()
    (gx,) = torch.autograd.grad(r.apply(leaf, pos.cuda(), transpose=transpose), leaf, w, create_graph=True)
    (gw,) = torch.autograd.grad(gx, w, torch.ones_like(gx))
    assert torch.equal(gw, r.apply(torch.ones_like(leaf), pos.cuda(), transpose=transpose))
    with torch.no_grad():
        assert not r.apply(leaf, pos.cuda()).requires_grad


@pytest.mark.gpu
def test_a_recorded_rotation_on_another_stream_and_captured():
    d = 64
    r = binding.Rope(d)
    pos = torch.arange(300, dtype=torch.int32, device="cuda")
    x = torch.randn(300, 4, d, device="cuda")
    dy = torch.randn(300, 4, d, device="cuda")
    want = r.apply(dy, pos, transpose=True)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        leaf = x.clone().requires_grad_()
        r.apply(leaf, pos).backward(dy)
    side.synchronize()
    assert torch.equal(leaf.grad, want)
    static = x.clone().requires_grad_()
    with torch.cuda.stream(side):
        for _ in range(2):
            static.grad = None
            r.apply(static, pos).backward(dy)
    torch.cuda.current_stream().wait_stream(side)
    static.grad = None
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y = r.apply(static, pos)
        y.backward(dy)
    for _ in range(2):
        with torch.no_grad():
            static.mul_(1.5)
            dy.mul_(0.5)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(y.detach(), r.apply(static.detach(), pos))
        assert torch.equal(static.grad, r.apply(dy, pos, transpose=True))


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_positions_past_31_bits_rotate_q(dtype):
    """start + i of rows that have no place may pass 2^31: q is rotated by the sum, not by what 32 bits leave of
    it. The reference's angle, position times theta in float64, is off by 2^-21 at theta = 1; here the turns are
    reduced in integers of 2^-64."""
    lay = Layout([0], [6], 1, 64, dtype=dtype, hq=2)
    io = binding.KVCacheIO(lay.problem)
    r = binding.Rope(64)
    start = 2 ** 31 - 3
    q, k = lay.normal(6, 2, 64), lay.normal(6, 1, 64)
    kc = lay.cache().cuda()
    before = kc.clone()
    out = io.write(k.cuda(), k.cuda(), kc, kc.clone(), None, lay.row_offsets.cuda(),
                   torch.tensor([start], dtype=torch.int32, device="cuda"), rope=r, q=q.cuda())
    assert torch.equal(kc, before)
    theta = r.frequencies()
    c, s = torch.zeros(6, 1, 32, dtype=torch.float64), torch.zeros(6, 1, 32, dtype=torch.float64)
    for i in range(6):
        for j, t in enumerate(theta):
            turn = Fraction(t) / Fraction(2 * math.pi)
            # theta / (2 pi) in double is off by 2^-53 of itself, 2 pi by 2^-53: times 2^31 turns, 2^-21
            a = float(((start + i) * turn) % 1) * 2 * math.pi
            c[i, 0, j], s[i, 0, j] = math.cos(a), math.sin(a)
    x = q.double()
    want = torch.cat([c * x[..., :32] - s * x[..., 32:], s * x[..., :32] + c * x[..., 32:]], -1)
    size = (x[..., :32].abs() + x[..., 32:].abs()).repeat(1, 1, 2)
    tol = size * (4e-7 + 3 * 2.0 ** -24 + 2.0 ** 31 * 2 * math.pi * 2.0 ** -51) + want.abs() * half_step(x.dtype)
    tol = tol + want.abs() * half_step(TORCH[dtype]) * 1.001
    assert ((out.cpu().double() - want).abs() <= tol).all()


@pytest.mark.gpu
@pytest.mark.parametrize("dtype,kv,hkv,d", [("bf16", "e4m3", 1, 64), ("bf16", "bf16", 1, 64), ("f32", "f32", 1, 64),
                                            ("bf16", "e4m3", 3, 64), ("bf16", "e4m3", 5, 128)])
def test_reads_of_short_and_odd_rows_at_every_length(dtype, kv, hkv, d):
    """Rows of 4 items and more, one tensor and both, row counts around a warp's and a block's items."""
    for rows in (1, 2, 31, 32, 33, 255, 256, 257, 1023, 1025):
        lay = Layout([5, 40], [rows, 3], hkv, d, page=8, dtype=dtype, kv=kv, before=1, behind=2, seed=rows)
        io = binding.KVCacheIO(lay.problem)
        kc, vc = lay.cache(), lay.cache()
        place = (lay.table.cuda(), lay.row_offsets.cuda(), lay.start.cuda())
        member = torch.tensor([b >= 0 for b in lay.row_seq])
        z = torch.tensor([lay.cache_row(b, t) for b, t in zip(lay.row_seq, lay.row_pos) if b >= 0])
        for which in ((0,), (1,), (0, 1)):
            src = [(kc, vc)[i].cuda() if i in which else None for i in range(2)]
            out = [torch.full((lay.rows, hkv, d), 9.0, dtype=TORCH[dtype], device="cuda") if i in which else None
                   for i in range(2)]
            io.read(*src, *place, *out)
            for i, scale in zip(range(2), (lay.k_scale, lay.v_scale)):
                if i in which:
                    want = (kc, vc)[i].reshape(-1, hkv, d)[z]
                    if kv == "e4m3":
                        want = (want.view(torch.float8_e4m3fn).float() * torch.tensor(scale)).to(TORCH[dtype])
                    assert torch.equal(out[i].cpu()[member], want) and (out[i].cpu()[~member] == 9.0).all()


@pytest.mark.gpu
@pytest.mark.parametrize("dtype,kv", KINDS)
def test_q_is_rotated_in_place_beside_k_and_v(dtype, kv):
    """q, k and v as parts of one projection's rows, q rotated where it lies: the same as into a tensor of its own,
    and k and v keep their values."""
    lay = Layout([30, 4], [50, 3], 2, 64, page=16, hq=8, dtype=dtype, kv=kv)
    io = binding.KVCacheIO(lay.problem)
    r = binding.Rope(64)
    wide = lay.normal(lay.rows, 12, 64).cuda()
    kept = wide.clone()
    place = (lay.table.cuda(), lay.row_offsets.cuda(), lay.start.cuda())
    a, b = ([lay.cache().cuda().zero_() for _ in range(2)] for _ in range(2))
    q = io.write(wide[:, 8:10], wide[:, 10:], *a, *place, rope=r, q=wide[:, :8])
    same = io.write(wide[:, 8:10], wide[:, 10:], *b, *place, rope=r, q=wide[:, :8], q_out=wide[:, :8])
    assert same.data_ptr() == wide.data_ptr() and torch.equal(same, q)
    assert torch.equal(wide[:, 8:], kept[:, 8:]) and all(torch.equal(x, y) for x, y in zip(a, b))
    with pytest.raises(binding.DecodeAttnError):
        io.write(wide[:, 8:10], wide[:, 10:], *b, *place, rope=r, q=kept[:, :8], q_out=wide[:, 2:10])
