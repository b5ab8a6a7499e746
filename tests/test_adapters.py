"""Low-rank adapters of many requests: refusals on the CPU, results on the GPU against plain float64 forms."""
import weakref

import pytest
import torch

from _rows import TORCH, half_step
from decode_attention_attn_gb300 import binding, build as lib_build

A = 0x10000000   # an aligned address that no refused call dereferences


@pytest.fixture(scope="module", autouse=True)
def built():
    lib_build.build()


# ---- CPU: refusals --------------------------------------------------------------------------
def test_apply_refuses_bad_arguments():
    P = 1 << 24

    def call(cfg=(), **kw):
        config = binding.da_adapter_config(2, 256, 2, (binding.ctypes.c_int * 4)(128, 64, 0, 0), 16)
        for k, v in dict(cfg).items():
            setattr(config, k, v if k != "out_sizes" else (binding.ctypes.c_int * 4)(*v))
        args = binding.da_adapter_args(A, A + P, A + 2 * P, A + 3 * P, A + 4 * P, A + 5 * P, A + 6 * P, A + 7 * P, 9, 4, 3,
                                       256, 192, 192, None)
        for k, v in kw.items():
            assert hasattr(args, k)
            setattr(args, k, v)
        with pytest.raises(binding.DecodeAttnError) as e:
            binding.decode_attn_adapters_apply(config, args)
        return e.value.code

    for cfg, code in ((dict(dtype=3), -2), (dict(dtype=-1), -2), (dict(width=0), -1), (dict(width=(1 << 20) + 1), -2),
                      (dict(parts=0), -1), (dict(parts=5), -2), (dict(rank=12), -2), (dict(rank=256), -2), (dict(rank=0), -2),
                      (dict(out_sizes=(128, 0, 0, 0)), -1), (dict(out_sizes=(128, (1 << 20) + 1, 0, 0)), -2)):
        assert call(cfg) == code, cfg
    for name in ("x", "y", "out", "a", "b", "row_offsets", "adapter_ids"):
        assert call(**{name: None}) == -1, name
    assert call(rows=-1) == -1 and call(batch=0) == -1 and call(adapters=0) == -1
    assert call(batch=16385) == -2 and call(adapters=8193) == -2
    for name, by in (("x", 1), ("y", 1), ("out", 1), ("a", 8), ("b", 2), ("scales", 2), ("row_offsets", 1), ("adapter_ids", 2)):
        assert call(**{name: A + 9 * P + by}) == -1, name
    # rows on one another, results over inputs
    assert call(out_row_stride=191) == -1 and call(out_row_stride=0) == -1 and call(out_row_stride=-192) == -1
    assert call(out=A + P, out_row_stride=384) == -1 and call(out=A + P + 64) == -1
    for i in (0, 3, 4, 5, 6, 7):
        assert call(out=A + i * P) == -1, i
    assert call(workspace=A + 9 * P + 16, workspace_bytes=4096) == -1
    assert call(workspace=A + 2 * P + 256, workspace_bytes=4096) == -1      # over the results
    # no rows: nothing is enqueued, no pointer is looked at
    config = binding.da_adapter_config(2, 256, 1, (binding.ctypes.c_int * 4)(128, 0, 0, 0), 16)
    binding.decode_attn_adapters_apply(config, binding.da_adapter_args(*[None] * 8, 0, 1, 1))
    with pytest.raises(binding.DecodeAttnError):
        binding._check(binding.lib().decode_attn_adapters_apply(None, None), "adapters")


def test_the_workspace_by_widths_rows_and_rank():
    def size(rows, dtype=2, width=4096, sizes=(4096, 1024, 1024, 0), parts=3, rank=64):
        config = binding.da_adapter_config(dtype, width, parts, (binding.ctypes.c_int * 4)(*sizes), rank)
        return binding.decode_attn_adapters_workspace(config, rows)

    assert size(8000) == size(8000, width=8192) > size(4000) > 256       # by rows, parts and rank
    assert size(8000, sizes=(8192, 8192, 8192, 0)) == size(8000) == size(8000, dtype=1)
    assert size(1023) == size(0) == size(8000, dtype=0) == size(8000, rank=128) == 0
    assert size(1100, width=256, sizes=(64, 64, 64, 0)) == size(2000, rank=8) == 0   # few weights: short launches
    for kw in (dict(rows=-1), dict(width=0), dict(parts=0), dict(parts=5), dict(rank=0), dict(rank=-8)):
        with pytest.raises(binding.DecodeAttnError) as e:
            size(**{"rows": 8000, **kw})
        assert e.value.code == -1


def test_wrapper_refuses_bad_tensors():
    for args in ((0, [8], 8), (64, [], 8), (64, [8] * 5, 8), (64, [8, 0], 8), (64, [8], 12)):
        with pytest.raises(ValueError):
            binding.Adapters(*args)
    with pytest.raises(ValueError):
        binding.Adapters(64, [8], 8, "f64")
    ad = binding.Adapters(64, [24, 8], 8, "f32")
    ok = dict(x=torch.zeros(5, 64), y=torch.zeros(5, 32), a=torch.zeros(3, 16, 64), b=torch.zeros(3, 32, 8),
              scales=torch.zeros(3), row_offsets=torch.zeros(3, dtype=torch.int32), adapter_ids=torch.zeros(2, dtype=torch.int32))
    bad = [dict(x=torch.zeros(5, 65)), dict(x=torch.zeros(4, 64)), dict(x=torch.zeros(5, 64).half()), dict(x=torch.zeros(64, 5).t()),
           dict(y=torch.zeros(5, 31)), dict(out=torch.zeros(4, 32)), dict(out=torch.zeros(5, 32).half()),
           dict(a=torch.zeros(3, 8, 64)), dict(a=torch.zeros(3, 16, 64).half()), dict(a=torch.zeros(3, 16, 128)[..., ::2]),
           dict(b=torch.zeros(2, 32, 8)), dict(b=torch.zeros(3, 32, 16)), dict(scales=torch.zeros(2)),
           dict(scales=torch.zeros(3).half()), dict(row_offsets=torch.zeros(4, dtype=torch.int32)),
           dict(adapter_ids=torch.zeros(2)), dict(adapter_ids=torch.zeros(0, dtype=torch.int32), row_offsets=torch.zeros(1, dtype=torch.int32))]
    for kw in bad:
        with pytest.raises(ValueError):
            ad.apply(**{**ok, **kw})
    with pytest.raises(ValueError, match="CUDA"):
        ad.apply(**ok)
    for name in ("x", "y", "a", "b"):
        with pytest.raises(ValueError, match="gradient"):
            ad.apply(**{**ok, name: ok[name].clone().requires_grad_()})


# ---- the plain form -------------------------------------------------------------------------
class Step:
    """Requests' rows and adapters, what the product is in 64 bits, and what a result may be off by."""

    def __init__(self, lens, ids, width, outs, rank, adapters, dtype, before=0, behind=0, seed=0, x_gain=1.0, x_pad=0,
                 y_pad=0, shift=0):
        g = torch.Generator().manual_seed(seed + width + rank)
        self.t, self.outs, self.rank = TORCH[dtype], outs, rank
        rows, columns = before + sum(lens) + behind, sum(outs)

        def strided(rows, n, pad, gain=1.0):
            flat = torch.zeros(shift + rows * (n + pad), dtype=self.t)
            flat[shift:].view(rows, n + pad).copy_(gain * torch.randn(rows, n + pad, generator=g))
            return flat.cuda()[shift:].view(rows, n + pad)[:, :n]

        self.x, self.y = strided(rows, width, x_pad, x_gain), strided(rows, columns, y_pad)
        self.a = (torch.randn(adapters, len(outs) * rank, width, generator=g) / width ** 0.5).to(self.t).cuda()
        self.b = (0.5 * torch.randn(adapters, columns, rank, generator=g) / rank ** 0.5).to(self.t).cuda()
        self.scales = (0.5 + torch.rand(adapters, generator=g)).cuda()
        offs = [before]
        for n in lens:
            offs.append(offs[-1] + n)
        self.offsets = torch.tensor(offs, dtype=torch.int32).cuda()
        self.ids = torch.tensor(ids, dtype=torch.int32).cuda()
        self.of = [-1] * rows
        self.member = torch.zeros(rows, dtype=torch.bool)
        for b, n in enumerate(lens):
            for r in range(offs[b], offs[b + 1]):
                self.of[r] = ids[b] if 0 <= ids[b] < adapters else -1
                self.member[r] = True
        self.handle = binding.Adapters(width, outs, rank, dtype)
        self.found = None

    def apply(self, out=None, long=False, **kw):
        """long: with a workspace whatever the widths (its size is that of the widest)."""
        if long:
            c = self.handle.config
            wide = binding.da_adapter_config(c.dtype, 1 << 20, c.parts, c.out_sizes, c.rank)
            rows = self.x.shape[0]
            size = binding.decode_attn_adapters_workspace(wide, rows)
            out = torch.empty_like(self.y) if out is None else out
            assert size
            stream = kw.get("stream") or torch.cuda.current_stream()
            with torch.cuda.stream(stream):
                ws = torch.zeros(size, dtype=torch.uint8, device="cuda")
            binding.decode_attn_adapters_apply(c, binding.da_adapter_args(
                self.x.data_ptr(), self.y.data_ptr(), out.data_ptr(), self.a.data_ptr(), self.b.data_ptr(),
                self.scales.data_ptr(), self.offsets.data_ptr(), self.ids.data_ptr(), rows, self.ids.numel(),
                self.a.shape[0], self.x.stride(0), self.y.stride(0), out.stride(0), ws.data_ptr(), size,
                stream.cuda_stream))
            self.found = ws[:4]
            return out
        return self.handle.apply(self.x, self.y, self.a, self.b, self.scales, self.offsets, self.ids, out=out, **kw)

    def want(self):
        """(result, bound). Of a low-rank number: a sum of width products, each exact (fp32: within 2^-20, two tf32
        parts of each factor without their smallest product), added 8 or 16 at a time, each addition within 2^-23 of
        the sum of magnitudes, then 8 warps and 8 CTAs. As an operand within 2^-17 (bf16 pairs) or 2^-20 (f16, tf32
        pairs); rank more products, added twice or three times 8 at a time."""
        width, rank = self.x.shape[1], self.rank
        f32 = self.t is torch.float32
        e1 = (3 * (width // 8 + 1) + 16 if f32 else width // 16 + 17) * 2.0 ** -23 + (2.0 ** -20 if f32 else 0)
        e2 = (3 * (rank // 8 + 1)) * 2.0 ** -23 + (2.0 ** -17 if self.t is torch.bfloat16 else 2.0 ** -20)
        want, off = self.y.double().clone(), torch.zeros_like(self.y, dtype=torch.float64)
        of = torch.tensor(self.of, device="cuda")
        for a in set(self.of) - {-1}:
            rows = (of == a).nonzero()[:, 0]
            x, at = self.x[rows].double(), 0
            for k, w in enumerate(self.outs):
                down = self.a[a, k * rank:(k + 1) * rank].double()
                up = self.b[a, at:at + w].double()
                low, mag = x @ down.T, x.abs() @ down.abs().T
                c = float(self.scales[a])
                want[rows, at:at + w] += c * (low @ up.T)
                most = low.abs().amax(1, keepdim=True)        # (f16: less than 2^-32 of the row's largest is cut off)
                off[rows, at:at + w] = c * ((e1 * mag + e2 * low.abs() + 2.0 ** -32 * most) @ up.abs().T)
                at += w
        fused = 2.0 ** -23 * (want.abs() + self.y.double().abs())
        bound = off * 1.01 + fused + want.abs() * half_step(self.t) + (2.0 ** -25 if self.t is torch.float16 else 0)
        return want, bound

    def check(self, got, before=None):
        want, bound = self.want()
        err = (got.double() - want).abs()
        m = self.member.cuda()
        assert (err[m] <= bound[m]).all(), float((err[m] / bound[m]).max())
        assert self.found is None or not self.found.any()
        if before is not None:
            assert torch.equal(got[~m], before[~m])


CASES = {   # lens, ids
    "one": ([1], [0]),
    "each": ([1] * 7, [3, 0, 4, 1, 2, 5, 6]),
    "shared": ([1, 3, 2, 1, 40, 1], [2, 2, 2, 2, 2, 2]),
    "bare": ([4, 1, 0, 2, 5], [-1, 1, 1, 7, 900]),
    "ragged": ([0, 17, 0, 0, 1, 33, 16, 64, 2], [1, 0, 1, 2, 1, 0, -1, 1, 0]),
    "prompts": ([300, 77, 129], [1, 0, 1]),
    "none": ([3, 2], [-1, -2]),
}


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("name", list(CASES))
@pytest.mark.parametrize("width,outs,rank", [(256, [128, 64], 16), (4096, [512, 128, 128], 8), (64, [8], 64), (1000, [40, 8, 16, 104], 32),
                                             (512, [96, 32], 128)])
def test_adapters(dtype, name, width, outs, rank):
    lens, ids = CASES[name]
    s = Step(lens, ids, width, outs, rank, 7, dtype, before=2, behind=3)
    before = torch.randn_like(s.y)
    out = before.clone()
    assert s.apply(out) is out
    s.check(out, before)
    # in place
    y0 = s.y.clone()
    want, bound = s.want()
    s.apply(s.y)
    m = s.member.cuda()
    assert ((s.y.double() - want).abs()[m] <= bound[m]).all() and torch.equal(s.y[~m], y0[~m])
    assert torch.equal(s.y[m], out[m])


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("name", ["ragged", "prompts"])
@pytest.mark.parametrize("width,outs,rank,x_pad,y_pad,shift", [
    (1001, [99, 7], 16, 0, 0, 0), (64, [5, 1, 1, 3], 8, 3, 1, 1), (256, [64, 65], 64, 0, 8, 0), (255, [64, 64], 32, 0, 0, 0),
    (256, [128], 16, 8, 16, 8), (256, [128], 16, 8, 16, 3), (1, [1], 128, 0, 0, 0), (7, [33], 32, 1, 0, 0),
    (1002, [34, 6], 16, 0, 0, 0), (1004, [36, 4], 8, 0, 4, 0), (100, [36, 52], 64, 4, 8, 4), (130, [64, 2], 32, 6, 2, 2),
    (256, [60], 16, 0, 4, 0), (252, [64], 16, 4, 0, 0)])
def test_odd_sizes_strides_and_alignment(dtype, name, width, outs, rank, x_pad, y_pad, shift):
    lens, ids = CASES[name]
    s = Step(lens, ids, width, outs, rank, 3, dtype, before=1, behind=1, x_pad=x_pad, y_pad=y_pad, shift=shift)
    out = torch.randn_like(s.y)
    before = out.clone()
    s.check(s.apply(out), before)
    wide = s.y._base.clone()
    s.apply(s.y)
    rows, n = s.y.shape
    same = torch.ones(rows, n + y_pad, dtype=torch.bool, device="cuda")
    same[s.member.cuda(), :n] = False
    assert torch.equal(s.y._base[shift:].view(rows, -1)[same], wide[shift:].view(rows, -1)[same])
    assert torch.equal(s.y._base[:shift], wide[:shift])


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("parts,rank", [(1, 8), (4, 128), (3, 64), (4, 64), (3, 128), (4, 8)])
@pytest.mark.parametrize("each", [1, 30, 200])
def test_every_tile_height_and_share(dtype, parts, rank, each):
    """Few, some and many rows an adapter, and low-rank columns for every split over the warps."""
    s = Step([each] * 3, [0, 1, 0], 320, [64 * (k + 1) for k in range(parts)], rank, 2, dtype)
    s.check(s.apply())


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["f16", "bf16", "f32"])
def test_many_requests_and_adapters(dtype):
    for batch, adapters, most in ((3000, 500, 3), (1, 8192, 40), (700, 3, 9), (16384, 2, 1)):
        g = torch.Generator().manual_seed(batch)
        lens = torch.randint(0, most + 1, (batch,), generator=g).tolist()
        ids = torch.randint(-1, adapters, (batch,), generator=g).tolist()
        lens[0], ids[0] = 2, adapters - 1
        s = Step(lens, ids, 64, [32], 8, adapters, dtype)
        s.check(s.apply())


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["f16", "bf16", "f32"])
def test_values_at_the_types_ends(dtype):
    """Low-rank numbers past f16's range, small ones beside them, rows of zeros, and rows that are not finite."""
    s = Step([5, 4], [0, 1], 512, [64, 32], 16, 2, dtype, x_gain=1000.0)
    s.b[0] *= 2.0 ** -9
    s.b[1] *= 2.0 ** -9
    s.a[0, :16] *= 512
    s.a[1, 3] *= 2.0 ** -12
    s.x[2] = 0
    out = s.apply()
    s.check(out)
    assert torch.equal(out[2], s.y[2])
    s.x[4, 7], s.x[7, 500] = float("inf"), float("nan")
    out2 = s.apply()
    assert not out2[4].isfinite().all() and out2[7].isnan().all()
    keep = [0, 1, 2, 3, 5, 6, 8]
    assert torch.equal(out2[keep], out[keep])


TALL = {   # lens, ids
    "prompts": ([1000, 1, 129, 128, 33], [1, 0, 2, 0, 1]),
    "mixed": ([1] * 40 + [31, 32, 64, 900, 0, 5, 300], [i % 3 for i in range(45)] + [-1, 1]),
    "bare": ([700, 600, 40, 10], [-1, 2, 9, 0]),
    "many": ([40] * 60, [i % 3 for i in range(60)]),
    "around": ([64, 63, 65, 127, 128, 129, 191, 193, 64, 64, 64], [0, 1, 2, 1, 0, 2, 1, 1, 1, 0, 1]),
}


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("name", list(TALL))
@pytest.mark.parametrize("width,outs,rank", [(256, [128, 64], 16), (1000, [520, 8, 136], 64), (520, [256], 8), (192, [40, 8, 16, 104], 32),
                                             (512, [96, 200], 128), (64, [8], 128), (2048, [384, 128], 32)])
def test_long_requests(dtype, name, width, outs, rank):
    """Steps that the tensor-core launches take a part of: tiles and blocks that end inside, every rank."""
    lens, ids = TALL[name]
    s = Step(lens, ids, width, outs, rank, 3, dtype, before=3, behind=60)
    before = torch.randn_like(s.y)
    out = before.clone()
    s.check(s.apply(out, long=True), before)
    m = s.member.cuda()
    y0 = s.y.clone()
    s.apply(s.y, long=True)
    assert torch.equal(s.y[m], out[m]) and torch.equal(s.y[~m], y0[~m])


@pytest.mark.gpu
@pytest.mark.parametrize("dtype,outs", [("bf16", [64, 24]), ("f16", [33]), ("f32", [5])])
def test_many_rows_without_an_adapter(dtype, outs):
    """More of them than the launch's CTAs take in one go, beside ones with one, with and without a workspace."""
    s = Step([9000, 20, 6000, 1, 0], [-1, 1, 5, 0, 1], 64, outs, 16, 2, dtype, before=1, behind=2)
    before = torch.randn_like(s.y)
    out = before.clone()
    s.check(s.apply(out), before)
    if dtype == "bf16":
        s.check(s.apply(before.clone(), long=True), before)


@pytest.mark.gpu
def test_long_requests_of_strided_rows_repeat_on_streams_and_in_graphs():
    s = Step([700, 400, 3], [1, 0, 1], 264, [96, 64], 16, 2, "bf16", before=1, behind=1, x_pad=8, y_pad=16, shift=8)
    wide = s.y._base.clone()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    out = s.apply(stream=side, long=True)
    side.synchronize()
    s.check(out)
    m = s.member.cuda()
    assert all(torch.equal(s.apply(long=True)[m], out[m]) for _ in range(3))
    # two at once
    for _ in range(4):
        a = s.apply(stream=side, long=True)
        b = s.apply(long=True)
        torch.cuda.synchronize()
        assert torch.equal(a[m], out[m]) and torch.equal(b[m], out[m])
    graph = torch.cuda.CUDAGraph()
    held = torch.empty_like(out)
    with torch.cuda.graph(graph):
        s.apply(held, long=True)
    for ids in ([0, 0, 0], [-1, 1, 0], [1, 1, 1]):
        s.ids.copy_(torch.tensor(ids, dtype=torch.int32))
        s.x.copy_(torch.randn(s.x.shape))
        s.of = [-1] + [a for n, a in zip([700, 400, 3], ids) for _ in range(n)] + [-1]
        graph.replay()
        s.check(held)
    rows, n = s.y.shape
    s.apply(s.y, long=True)
    same = torch.ones(rows, n + 16, dtype=torch.bool, device="cuda")
    same[m, :n] = False
    assert torch.equal(s.y._base[8:].view(rows, -1)[same], wide[8:].view(rows, -1)[same])


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["f16", "bf16"])
def test_long_requests_with_values_at_the_types_ends(dtype):
    s = Step([1100, 60], [0, 1], 512, [64, 32], 16, 2, dtype, x_gain=1000.0)
    s.b[:] *= 2.0 ** -9
    s.a[0, :16] *= 512
    s.a[1, 3] *= 2.0 ** -12
    s.x[2] = 0
    out = s.apply(long=True)
    s.check(out)
    assert torch.equal(out[2], s.y[2])
    s.x[4, 7], s.x[1130, 500] = float("inf"), float("nan")
    out2 = s.apply(long=True)
    assert not out2[4].isfinite().all() and out2[1130].isnan().all()
    keep = torch.ones(1160, dtype=torch.bool)
    keep[[4, 1130]] = False
    assert torch.equal(out2[keep.cuda()], out[keep.cuda()])


@pytest.mark.gpu
def test_workspaces_of_long_steps():
    """Without one a long step is answered all the same, a short one is refused, and nothing is found; where the
    weights are few there is none."""
    few = binding.Adapters(256, [64, 64], 32)
    assert binding.decode_attn_adapters_workspace(few.config, 1290) == 0 < \
        binding.decode_attn_adapters_workspace(binding.Adapters(1 << 20, [64, 64], 32).config, 1290)
    s = Step([1200, 90], [1, 0], 4096, [2048] * 4, 64, 2, "bf16")
    size = binding.decode_attn_adapters_workspace(s.handle.config, 1290)
    assert size > 256 and binding.decode_attn_adapters_workspace(s.handle.config, 1023) == 0
    ws = torch.zeros(size, dtype=torch.uint8, device="cuda")
    out = torch.empty_like(s.y)
    args = binding.da_adapter_args(s.x.data_ptr(), s.y.data_ptr(), out.data_ptr(), s.a.data_ptr(), s.b.data_ptr(),
                                   s.scales.data_ptr(), s.offsets.data_ptr(), s.ids.data_ptr(), 1290, 2, 2, 4096, 8192, 8192,
                                   ws.data_ptr(), size, torch.cuda.current_stream().cuda_stream)
    binding.decode_attn_adapters_apply(s.handle.config, args)
    s.check(out)
    binding.decode_attn_adapters_check_status(ws.data_ptr())
    args.workspace_bytes = size - 1
    with pytest.raises(binding.DecodeAttnError) as e:
        binding.decode_attn_adapters_apply(s.handle.config, args)
    assert e.value.code == -3
    kept = binding.Adapters(4096, [2048] * 4, 64, findings=True)
    want, bound = s.want()
    for n in (1290, 1200, 9):
        got = kept.apply(s.x[:n], s.y[:n], s.a, s.b, s.scales, s.offsets, s.ids)
        assert ((got.double() - want[:n]).abs() <= bound[:n]).all() and (n < 1290 or torch.equal(got, out))
        kept.check_status()
    assert kept.workspace_bytes == size
    with pytest.raises(ValueError):
        s.handle.check_status()
    args.workspace, args.workspace_bytes = None, 0
    out.zero_()
    binding.decode_attn_adapters_apply(s.handle.config, args)
    s.check(out)


@pytest.mark.gpu
def test_broadcast_rows_no_scales_and_four_dimensions():
    s = Step([30, 1], [1, 0], 128, [64], 8, 2, "bf16")
    s.x = s.x[:1].expand(31, 128)
    s.check(s.apply())
    s.scales[:] = 1
    got = s.handle.apply(s.x, s.y, s.a.view(2, 1, 8, 128), s.b, None, s.offsets, s.ids)
    s.check(got)
    empty = s.handle.apply(s.x[:0], s.y[:0], s.a, s.b, None, s.offsets, s.ids)
    assert empty.shape == (0, 64)
    # offsets that reach past the rows there are
    got = s.handle.apply(s.x[:9], s.y[:9], s.a, s.b, None, s.offsets, s.ids)
    want, bound = s.want()
    assert ((got.double() - want[:9]).abs() <= bound[:9]).all()


@pytest.mark.gpu
def test_offsets_past_32_bits():
    """Adapters more than 2^31 elements in, rows as far apart."""
    width, rank, adapters = 1 << 20, 128, 18
    handle = binding.Adapters(width, [32], rank, "bf16")
    a = torch.zeros(adapters, rank, width, dtype=torch.bfloat16, device="cuda")
    a[17, 127, 1048570], a[16, 0, 3] = 2.0, 3.0
    b = torch.zeros(adapters, 32, rank, dtype=torch.bfloat16, device="cuda")
    b[17, 31, 127], b[16, 0, 0] = 0.5, 4.0
    far = torch.zeros((1 << 31) + 64 + width, dtype=torch.bfloat16, device="cuda")
    x = far.as_strided((2, width), ((1 << 31) + 64, 1))
    x[0, 3], x[1, 1048570] = 1.5, 7.0
    y = torch.zeros(2, 32, dtype=torch.bfloat16, device="cuda")
    out = handle.apply(x, y, a, b, None, torch.tensor([0, 1, 2], dtype=torch.int32).cuda(),
                       torch.tensor([16, 17], dtype=torch.int32).cuda())
    want = torch.zeros(2, 32)
    want[0, 0], want[1, 31] = 18.0, 7.0
    assert torch.equal(out.cpu().float(), want)


@pytest.mark.gpu
def test_streams_graphs_and_repeats():
    s = Step([3, 1, 20, 6], [1, 0, 2, 1], 1024, [256, 64], 16, 3, "bf16")
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    out = s.apply(stream=side)
    side.synchronize()
    s.check(out)
    assert all(torch.equal(s.apply(), out) for _ in range(3))
    graph = torch.cuda.CUDAGraph()
    held = torch.empty_like(s.y)
    with torch.cuda.graph(graph):
        s.apply(held)
    for ids in ([0, 0, 0, 0], [2, -1, 1, 0], [1, 2, 2, 2]):
        s.ids.copy_(torch.tensor(ids, dtype=torch.int32))
        s.x.copy_(torch.randn(s.x.shape))
        s.of = [a for n, a in zip([3, 1, 20, 6], ids) for _ in range(n)]
        graph.replay()
        s.check(held)


LONG_RUNS = [   # width, outs, rank, rows: what a CTA of 152 has, of blocks of 128 columns, of segments (blocks of one
                # tile and part) and of units of the contraction (64 of a tile's width)
    (64, [128, 64, 128, 64], 8, 40000),     # 7.5 blocks, as many segments; 1.9 units, 1 a tile
    (192, [128, 64, 64, 64], 64, 26000),    # 5.1 blocks, as many segments; 3.8 units, 3 a tile
    (1000, [2048, 128, 128], 64, 6400),     # 7.1 blocks, 1.2 segments; 6.3 units, 16 a tile
    (520, [64], 128, 100000),               # 4.7 blocks, as many segments; 42.5 units, 9 a tile
    (328, [136, 1000], 32, 16000),          # 7.4 blocks, 1.5 segments; 4.4 units, 6 a tile
]


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("width,outs,rank,rows", LONG_RUNS)
def test_long_runs_of_the_tensor_core_launches(dtype, width, outs, rank, rows):
    """A CTA's run goes through its rings, accumulators and operands several times, over tiles and parts whose
    numbers are of other sizes (f16: with powers of two of their own), single blocks among them."""
    lens, sizes = [], [1000, 77, 640, 129, 64, 333, 1500, 63, 0, 200]
    while sum(lens) < rows:
        lens.append(sizes[len(lens) % len(sizes)])
    s = Step(lens, [i % 4 - (i % 7 == 6) for i in range(len(lens))], width, outs, rank, 3, dtype, before=5, behind=9)
    s.x.mul_(2.0 ** (torch.arange(s.x.shape[0], device="cuda") * 7 % 9 - 4)[:, None].to(s.t))
    for k in range(len(outs)):
        s.a[:, k * rank:(k + 1) * rank] *= 2.0 ** (3 * (k % 3) - 3)
    before = torch.randn_like(s.y)
    out = before.clone()
    s.check(s.apply(out, long=True), before)
    m = s.member.cuda()
    for _ in range(3):
        assert torch.equal(s.apply(long=True)[m], out[m])
    s.apply(s.y, long=True)
    assert torch.equal(s.y[m], out[m])


@pytest.mark.gpu
@pytest.mark.parametrize("where", ["x", "a", "b", "far"])
@pytest.mark.parametrize("width,outs,rank", [(64, [40, 24], 16), (257, [33], 8), (128, [64], 128)])
def test_infinities_in_fp32(width, outs, rank, where):
    """An infinity times a number that is exact in a part of it, or whose rest has the other sign, is an infinity."""
    s = Step([3, 20, 1], [0, 1, 0], width, outs, rank, 2, "f32")
    s.x.abs_()
    s.a.abs_()
    s.b.abs_().add_(2.0 ** -10)
    s.x[:, ::2] = 1.0                                   # (nothing left behind its first part)
    s.b[:, ::3] = 0.5
    for v in (float("inf"), -float("inf")):
        if where == "x":
            s.x[1, 5], s.x[7, 6] = v, -v
        elif where == "a":
            s.a[0, 3, 2], s.a[1, 1, 5] = v, -v
        elif where == "b":
            s.b[0, 4, 1], s.b[1, 7, rank - 1] = v, -v
        else:                                           # 2^-14 below the largest number there is, and small weights
            s.x[1, 5], s.a[:] = 3.4027e38 if v > 0 else -3.4027e38, 2.0 ** -100
        got, want = s.apply(), s.want()[0].float()
        assert not want.isnan().any() and (where == "far" or want.isinf().any())
        assert torch.equal(got.isinf(), want.isinf()) and torch.equal(got.sign()[want.isinf()], want.sign()[want.isinf()])
        assert not got.isnan().any()
        if where == "far":
            s.check(got)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("long", [False, True])
def test_an_infinite_low_rank_number_beside_large_ones(dtype, long):
    """Its columns are infinite, whatever the row's others are (which in f16 pass the operand's range unless they are
    taken by a power of two)."""
    s = Step([1100, 60] if long else [9, 3], [0, 1], 256, [64, 32], 16, 2, dtype, x_gain=1000.0)
    n = 1100 if long else 9
    s.b[:] *= 2.0 ** -9
    s.a[0] *= 512                                       # numbers up to 10^6
    s.x[:n, 7] = 1.0
    s.a[0, ::16, 7] = float("inf")                      # each part's first one
    s.b[0, :, 0] = s.b[0, :, 0].abs() + 0.5
    s.b[0, ::2, 0] *= -1
    got = s.apply(long=long)
    sign = torch.tensor([-1.0, 1.0], device="cuda").repeat(48)
    assert torch.equal(got[:n].float(), (sign * float("inf")).expand(n, 96))
    want, bound = s.want()
    assert torch.equal(want[:n].float(), got[:n].float())
    assert ((got.double() - want).abs() <= bound)[n:].all()


@pytest.mark.gpu
def test_a_captured_step_keeps_its_workspace_when_longer_ones_come():
    """Findings are kept of each; what the allocator gives out later is not the graph's."""
    s = Step([1200, 1400, 90], [1, 0, 1], 4096, [2048] * 4, 64, 2, "bf16")
    kept = binding.Adapters(4096, [2048] * 4, 64, findings=True)
    first = Step([1200, 90], [1, 0], 4096, [2048] * 4, 64, 2, "bf16")
    call = lambda t, **kw: kept.apply(t.x, t.y, t.a, t.b, t.scales, t.offsets, t.ids, **kw)
    first.check(call(first))
    held = torch.zeros_like(first.y)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call(first, out=held)
    ws = weakref.ref(kept.workspace)
    size = kept.workspace_bytes
    s.check(call(s))
    assert ws() is not None and kept.workspace is not ws() and kept.workspace_bytes >= 2 * size
    others = [torch.full((size,), 0x55, dtype=torch.uint8, device="cuda") for _ in range(4)]
    graph.replay()
    first.check(held)
    assert all((o == 0x55).all() for o in others)
    kept.check_status()
    ws()[:4] = torch.tensor([4, 0, 0, 0], dtype=torch.uint8)        # (what a wait that ran out leaves)
    with pytest.raises(binding.DecodeAttnError) as e:
        kept.check_status()
    assert e.value.code == -6
    kept.check_status()


def test_a_workspace_over_other_arguments_is_refused():
    P = 1 << 24
    config = binding.da_adapter_config(2, 256, 2, (binding.ctypes.c_int * 4)(128, 64, 0, 0), 16)
    for i in range(8):     # x, y, out, a, b, scales, row_offsets, adapter_ids
        args = binding.da_adapter_args(A, A + P, A + 2 * P, A + 3 * P, A + 4 * P, A + 5 * P, A + 6 * P, A + 7 * P, 2000, 4, 3,
                                       256, 192, 192, A + i * P, 1 << 20, None)
        with pytest.raises(binding.DecodeAttnError) as e:
            binding.decode_attn_adapters_apply(config, args)
        assert e.value.code == -1, i


@pytest.mark.gpu
def test_a_workspace_is_not_made_inside_a_capture():
    s = Step([1200, 90], [1, 0], 4096, [2048] * 4, 64, 2, "bf16")
    kept = binding.Adapters(4096, [2048] * 4, 64, findings=True)
    call = lambda **kw: kept.apply(s.x, s.y, s.a, s.b, s.scales, s.offsets, s.ids, **kw)
    held, side = torch.zeros_like(s.y), torch.cuda.Stream()
    for kw in ({}, {"stream": side}):
        graph = torch.cuda.CUDAGraph()
        with pytest.raises(ValueError, match="capture"):
            with torch.cuda.graph(graph, **kw):
                held.zero_()
                call(out=held, **kw)
        assert kept.workspace is None
    s.check(call())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call(out=held)
    graph.replay()
    s.check(held)
    kept.check_status()
