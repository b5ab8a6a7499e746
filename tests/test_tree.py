"""Attention for trees of drafted tokens: refusals on the CPU, results on the GPU against a plain
float64 form.

Tolerances. With an fp32 output the result is held to fp32 accumulation of exact products: K, q and V
enter the products exactly, a weight p is either fp32 or split into two 16-bit parts (2^-17 of it at
most is lost), exp2 is within 2^-22, its argument x = scale log2(e) q.k is off by 2^-22 of the sum of
|q k| terms. REL covers these for logits up to ~40 in size: |err| <= REL * sum_t p_t |v_t|, REL = 2^-15.
A 16-bit output adds half a step. Over an FP8 cache a 16-bit output takes its weights as one f16 each: half a
step is 2^-11 of a weight, or 2^-25 = 2^-11 * 2^-14 below f16's normal range, with the weights scaled so that
the largest is at least 1 (their sum too), so sum_t p_t |v_t| 2^-11 + 2^-11 2^-14 sum_t |v_t| is added. The log-sum-exp: 1e-5 * max(1, |lse|), as for the decode step."""
import math

import pytest
import torch

from _rows import Layout, TORCH, half_step
from decode_attention_attn_gb300 import binding, build as lib_build

A = 0x100000
REL = 2.0 ** -15
KINDS = [("f32", "f32"), ("f16", "f16"), ("bf16", "bf16"), ("bf16", "e4m3")]


@pytest.fixture(scope="module", autouse=True)
def built():
    lib_build.build()


def random_trees(lay, gen, hide=0.0):
    """One word a row: ancestors and itself in a random tree (a row may see nothing with `hide`)."""
    words = [-1] * lay.rows          # rows of no sequence hold all ones
    r0 = int(lay.row_offsets[0])
    for n in lay.new:
        of = []
        for i in range(n):
            parent = int(torch.randint(-1, i, (1,), generator=gen)) if i else -1
            of.append((of[parent] if parent >= 0 else 0) | 1 << i)
        for i in range(n):
            w = 0 if float(torch.rand(1, generator=gen)) < hide else of[i]
            # bits past the tree are ignored
            w |= (((1 << 64) - 1) >> n << n) if n < 64 else 0
            words[r0 + i] = w - (1 << 64) if w >= 1 << 63 else w
        r0 += n
    return torch.tensor(words, dtype=torch.int64)


def one_part(lay):
    """Whether a weight enters as one f16."""
    return lay.kv == "e4m3" and lay.problem.out_dtype != binding.DA_F32


def reference(lay, q, kc, vc, words, scale):
    """(out, lse, sum_t p |v|) in float64; rows of no sequence are NaN."""
    G = lay.hq // lay.hkv
    k_all, v_all = lay.values(kc, lay.k_scale), lay.values(vc, lay.v_scale)
    out = torch.full(q.shape, math.nan, dtype=torch.float64)
    lse = torch.full(q.shape[:2], math.nan, dtype=torch.float64)
    mag = out.clone()
    r0 = int(lay.row_offsets[0])
    for b, (ctx, n) in enumerate(zip(lay.held, lay.new)):
        if n:
            at = torch.tensor([lay.cache_row(b, t) for t in range(ctx + n)])
            k, v = k_all[at], v_all[at]
            for i in range(n):
                w = int(words[r0 + i]) if words is not None else (1 << i + 1) - 1
                seen = list(range(ctx)) + [ctx + j for j in range(n) if w >> j & 1]
                if not seen:
                    out[r0 + i], lse[r0 + i], mag[r0 + i] = 0.0, -math.inf, 0.0
                    continue
                ks = k[seen].repeat_interleave(G, 1)
                vs = v[seen].repeat_interleave(G, 1)
                x = torch.einsum("hd,thd->ht", q[r0 + i].double(), ks) * scale
                lse[r0 + i] = torch.logsumexp(x, -1)
                p = (x - lse[r0 + i][:, None]).exp()
                out[r0 + i] = torch.einsum("ht,thd->hd", p, vs)
                mag[r0 + i] = torch.einsum("ht,thd->hd", p, vs.abs())
                if one_part(lay):
                    mag[r0 + i] += 2.0 ** -14 * vs.abs().sum(0)
        r0 += n
    return out, lse, mag


def run(lay, q, kc, vc, words, scale, max_tree=None, fill=5.0, obj=None):
    t = obj or binding.TreeAttention(lay.problem, max_tree or max(max(lay.new), 1))
    out = torch.full((lay.rows, lay.hq, lay.d), fill, device="cuda",
                     dtype=t._cache.out_dtype)
    lse = torch.full((lay.rows, lay.hq), fill, device="cuda")
    t.run(q.cuda(), kc.cuda(), vc.cuda(), lay.table.cuda() if lay.page else None, lay.row_offsets.cuda(),
          lay.start.cuda(), None if words is None else words.cuda(), scale, out=out, out_lse=lse)
    return out.cpu(), lse.cpu(), t


def check(lay, got, lse, ref, fill=5.0):
    out, want_lse, mag = ref
    none = torch.tensor([b < 0 for b in lay.row_seq])
    assert (got[none] == fill).all() and (lse[none] == fill).all()
    got, lse, out, want_lse, mag = (x[~none].double() for x in (got, lse, out, want_lse, mag))
    empty = torch.isinf(want_lse)
    assert torch.equal(torch.isinf(lse), empty) and (got[empty] == 0).all()
    tol = mag * (REL + (2.0 ** -11 if one_part(lay) else 0))
    if lay.problem.out_dtype != binding.DA_F32:
        kind = torch.float16 if lay.problem.out_dtype == binding.DA_F16 else torch.bfloat16
        tol = tol + (out.abs() + tol) * half_step(kind) + (2.0 ** -25 if kind == torch.float16 else 0)
    bad = ~((got - out).abs() <= tol)
    assert not bad.any(), (bad.sum().item(), ((got - out).abs() / tol.clamp(min=1e-30)).max().item())
    err = (lse - want_lse)[~empty].abs()
    assert (err <= 1e-5 * want_lse[~empty].abs().clamp(min=1.0)).all(), err.max().item()


# ---- CPU: plans and refusals ------------------------------------------------------------------
def _prob(**kw):
    base = dict(batch=4, num_q_heads=32, num_kv_heads=8, head_dim=128, qkv_dtype="bf16",
                out_dtype="bf16", paged=True, page_size=16, max_blocks_per_seq=64,
                num_physical_blocks=256, num_sms=152)
    return binding.make_problem(**{**base, **kw})


@pytest.mark.parametrize("kw,tree,code", [
    (dict(), 0, -1), (dict(), 65, -1), (dict(), -3, -1),
    (dict(mode="unified"), 8, -2), (dict(mode="unified_local"), 8, -2),
    (dict(mode="unified", range_lo=1.0, range_hi=1.0), 8, -1),
    (dict(debug_stall_stage=1), 8, -1), (dict(batch=0), 8, -1), (dict(head_dim=96), 8, -2),
    (dict(num_q_heads=24), 8, -2), (dict(page_size=12), 8, -2),
    (dict(kv_dtype="e4m3", k_scale=0.0), 8, -1),
])
def test_plan_refuses(kw, tree, code):
    with pytest.raises(binding.DecodeAttnError) as e:
        binding.decode_attn_tree_plan(_prob(**kw), tree)
    assert e.value.code == code


@pytest.mark.parametrize("dtype,kv", KINDS)
@pytest.mark.parametrize("hq,hkv,d,tree", [(32, 8, 128, 64), (8, 8, 64, 1), (16, 2, 128, 13), (4, 2, 64, 64)])
def test_plan_info(dtype, kv, hq, hkv, d, tree):
    plan, ws = binding.decode_attn_tree_plan(
        _prob(num_q_heads=hq, num_kv_heads=hkv, head_dim=d, qkv_dtype=dtype, out_dtype=dtype, kv_dtype=kv), tree)
    i = binding.decode_attn_tree_plan_info(plan)
    rows = tree * hq // hkv
    assert i.row_tiles == -(-rows // i.tile_rows) and i.max_tree == tree
    assert i.workspace_bytes == ws and i.smem_bytes <= 232448
    assert 1 <= i.grid_ctas <= 2 * 152 and i.grid_ctas >= i.row_tiles
    binding.decode_attn_tree_destroy(plan)


def test_run_refuses_bad_arguments():
    plan, ws = binding.decode_attn_tree_plan(_prob(), 8)
    flat, _ = binding.decode_attn_tree_plan(_prob(paged=False, max_seq_len=64), 8)

    def call(plan=plan, **kw):
        args = binding.da_tree_args(A, A, A, A, A, A, A, 4, 0.1, A + 65536, A, A, ws, None)
        for k, v in kw.items():
            assert hasattr(args, k)
            setattr(args, k, v)
        with pytest.raises(binding.DecodeAttnError) as e:
            binding.decode_attn_tree_run(plan, args)
        return e.value.code

    for name in ("q", "k_cache", "v_cache", "block_table", "row_offsets", "ctx_lens", "out", "workspace"):
        assert call(**{name: None}) == -1, name
    assert call(rows=-1) == -1 and call(scale=math.nan) == -1 and call(scale=math.inf) == -1
    for name, off in (("q", 8), ("k_cache", 8), ("v_cache", 2), ("out", 8), ("out_lse", 2), ("tree_mask", 4),
                      ("row_offsets", 2), ("ctx_lens", 1), ("block_table", 2), ("workspace", 128)):
        assert call(**{name: A + off}) == -1, name
    assert call(out=A) == -1 and call(out=A + 4 * 32 * 128 * 2 - 16) == -1      # over q
    assert call(scale=3e38) == -1                            # times log2(e): no float
    assert call(workspace_bytes=ws - 1) == -3
    assert call(flat) == -1                                  # a table for a contiguous cache
    L = binding.lib()
    assert L.decode_attn_tree_run(plan, None) == -1 and L.decode_attn_tree_run(None, None) == -1
    assert L.decode_attn_tree_plan(None, 1, None, None) == -1
    assert L.decode_attn_tree_plan_info(plan, None) == -1
    assert L.decode_attn_tree_check_status(plan, None, None) == -1
    assert L.decode_attn_tree_workspace_init(plan, A, ws - 1, None) == -3
    assert L.decode_attn_tree_workspace_init(plan, A + 16, ws, None) == -1
    L.decode_attn_tree_destroy(None)
    # no rows: nothing is enqueued
    binding.decode_attn_tree_run(plan, binding.da_tree_args(None, None, None, A, A, A, None, 0, 0.1, None, None,
                                                            A, ws, None))
    for p in (plan, flat):
        binding.decode_attn_tree_destroy(p)


# ---- GPU --------------------------------------------------------------------------------------
SHAPES = [   # hq, hkv, d, page
    (8, 8, 64, 0), (8, 4, 128, 16), (16, 4, 128, 0), (16, 2, 64, 8), (4, 1, 128, 64), (12, 3, 128, 256),
]
LENGTHS = {
    "one": dict(held=[0], new=[1]),
    "short": dict(held=[0, 1, 5, 0], new=[1, 1, 3, 7]),
    "edges": dict(held=[127, 128, 129, 63, 64, 60, 250], new=[1, 5, 2, 1, 1, 8, 12]),
    "ragged": dict(held=[300, 0, 17, 1000, 9], new=[5, 0, 33, 2, 64], before=3, behind=4),
    "long": dict(held=[5000], new=[9]),
    "wide": dict(held=[513, 90], new=[64, 63]),
}


@pytest.mark.gpu
@pytest.mark.parametrize("dtype,kv", KINDS)
@pytest.mark.parametrize("hq,hkv,d,page", SHAPES)
@pytest.mark.parametrize("name", list(LENGTHS))
def test_tree(dtype, kv, hq, hkv, d, page, name):
    lay = Layout(**LENGTHS[name], hkv=hkv, d=d, page=page, hq=hq, dtype=dtype, kv=kv, seed=11)
    kc, vc = lay.cache(), lay.cache()
    if kv == "e4m3":     # random codes are huge; rows of N(0, 1) / scale instead
        kc, vc = ((torch.randn(lay.shape, generator=lay.gen) / s).clamp(-448, 448).to(torch.float8_e4m3fn)
                  .view(torch.uint8) for s in (lay.k_scale, lay.v_scale))
    q = lay.normal(lay.rows, hq, d)
    words = random_trees(lay, lay.gen, hide=0.15)
    scale = 1 / math.sqrt(d)
    out, lse, t = run(lay, q, kc, vc, words, scale, max_tree=64 if name == "ragged" else None)
    check(lay, out, lse, reference(lay, q, kc, vc, words, scale))
    t.check_status()
    if name in ("short", "edges"):
        out, lse, _ = run(lay, q, kc, vc, None, scale)
        check(lay, out, lse, reference(lay, q, kc, vc, None, scale))


def fill_normal(lay):
    """K and V rows of N(0, 1) in the cache's storage."""
    if lay.kv != "e4m3":
        return lay.normal(*lay.shape), lay.normal(*lay.shape)
    return tuple((torch.randn(lay.shape, generator=lay.gen) / s).clamp(-448, 448).to(torch.float8_e4m3fn)
                 .view(torch.uint8) for s in (lay.k_scale, lay.v_scale))


@pytest.mark.gpu
@pytest.mark.parametrize("dtype,kv", KINDS)
@pytest.mark.parametrize("sms", [1, 3, 7, 40])
@pytest.mark.parametrize("hq,hkv,d", [(8, 8, 64), (32, 4, 128), (12, 3, 128)])
def test_tree_on_few_ctas(dtype, kv, sms, hq, hkv, d):
    """Plans for few SMs: many pieces a CTA, groups that start, end and cross in every way, row tiles and heads
    that do not divide the CTAs."""
    lay = Layout([700, 0, 129, 5, 1300, 64, 2], [9, 33, 0, 64, 1, 20, 7], hkv, d, page=16, hq=hq, dtype=dtype,
                 kv=kv, num_sms=sms, seed=sms)
    kc, vc = fill_normal(lay)
    q, words = lay.normal(lay.rows, hq, d), random_trees(lay, lay.gen, hide=0.1)
    out, lse, t = run(lay, q, kc, vc, words, 0.1)
    check(lay, out, lse, reference(lay, q, kc, vc, words, 0.1))
    t.check_status()


@pytest.mark.gpu
@pytest.mark.parametrize("kv", ["bf16", "e4m3"])
def test_offsets_past_32_bits(kv):
    """A pool of more than 2^31 elements: pages at its far end."""
    page, hkv, d, hq = 64, 8, 128, 32
    pool = 2 ** 31 // (page * hkv * d) + 7
    fp8 = kv == "e4m3"
    prob = binding.make_problem(batch=2, num_q_heads=hq, num_kv_heads=hkv, head_dim=d, qkv_dtype="bf16",
                                out_dtype="f32", paged=True, page_size=page, max_blocks_per_seq=3,
                                num_physical_blocks=pool, kv_dtype=kv, k_scale=0.0125, v_scale=0.0125)
    kc, vc = (torch.zeros((pool, page, hkv, d), dtype=torch.uint8 if fp8 else torch.bfloat16, device="cuda")
              for _ in range(2))
    pages = torch.tensor([[pool - 1, pool - 3, 0], [pool - 2, 1, pool - 4]])
    small = Layout([150, 70], [6, 3], hkv, d, page=page, hq=hq, kv=kv, capacity=192, spare=0, k_scale=0.0125,
                   v_scale=0.0125, out_dtype="f32")
    sk, sv = fill_normal(small)
    for b in range(2):
        for i in range(3):
            if small.table[b, i] >= 0:
                kc[pages[b, i]], vc[pages[b, i]] = sk[small.table[b, i]].cuda(), sv[small.table[b, i]].cuda()
    q = small.normal(small.rows, hq, d)
    out, lse = binding.TreeAttention(prob, 6).run(q.cuda(), kc, vc, pages.int().cuda(), small.row_offsets.cuda(),
                                                  small.start.cuda(), None, 0.1)
    check(small, out.cpu(), lse.cpu(), reference(small, q, sk, sv, None, 0.1))


@pytest.mark.gpu
@pytest.mark.parametrize("dtype,kv", KINDS)
def test_a_chain_is_a_lower_triangular_mask_and_streams_are_taken(dtype, kv):
    lay = Layout([260, 3], [64, 11], 2, 64, page=8, hq=8, dtype=dtype, kv=kv)
    kc, vc = fill_normal(lay)
    q = lay.normal(lay.rows, 8, 64).cuda()
    words = [(1 << i + 1) - 1 for n in lay.new for i in range(n)]
    words = torch.tensor([w - (1 << 64) if w >> 63 else w for w in words]).cuda()
    t = binding.TreeAttention(lay.problem, 64)
    place = (kc.cuda(), vc.cuda(), lay.table.cuda(), lay.row_offsets.cuda(), lay.start.cuda())
    torch.cuda.synchronize()      # inputs of another stream: theirs to wait for; results are made on `side`
    side = torch.cuda.Stream()
    a = t.run(q, *place, None, 0.1, stream=side)
    b = t.run(q, *place, words, 0.1, stream=side)
    side.synchronize()
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


@pytest.mark.gpu
@pytest.mark.parametrize("dtype,kv", [("bf16", "bf16"), ("f16", "f16"), ("bf16", "e4m3")])
@pytest.mark.parametrize("d", [64, 128])
def test_tree_fp32_output(dtype, kv, d):
    """The unrounded result, to the fp32 bound."""
    lay = Layout([700, 33, 1290], [20, 64, 3], 2, d, page=16, hq=8, dtype=dtype, kv=kv, out_dtype="f32")
    kc, vc = lay.cache(), lay.cache()
    if kv == "e4m3":
        kc, vc = ((torch.randn(lay.shape, generator=lay.gen) / s).clamp(-448, 448).to(torch.float8_e4m3fn)
                  .view(torch.uint8) for s in (lay.k_scale, lay.v_scale))
    q = lay.normal(lay.rows, 8, d)
    words = random_trees(lay, lay.gen)
    out, lse, _ = run(lay, q, kc, vc, words, 0.1)
    check(lay, out, lse, reference(lay, q, kc, vc, words, 0.1))


@pytest.mark.gpu
@pytest.mark.parametrize("dtype,kv", KINDS)
@pytest.mark.parametrize("scale", [0.0, -0.3, 2.0])
def test_tree_scales(dtype, kv, scale):
    """Sharp, flat and negative logits: the running maximum moves by hundreds within a sequence. The logits'
    own fp32 error grows with them: 2^-22 of sum |q k| (about d/2 at N(0, 1)) times the scale."""
    lay = Layout([900, 40], [7, 12], 2, 64, page=16, hq=4, dtype=dtype, kv=kv, k_scale=0.0625, v_scale=0.125,
                 out_dtype="f32")
    kc, vc = lay.normal(*lay.shape), lay.normal(*lay.shape)
    if kv == "e4m3":
        kc, vc = ((x.float() / s).clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)
                  for x, s in ((kc, lay.k_scale), (vc, lay.v_scale)))
    q = lay.normal(lay.rows, 4, 64) * 2
    words = random_trees(lay, lay.gen)
    out, lse, _ = run(lay, q, kc, vc, words, scale)
    ref, ref_lse, mag = reference(lay, q, kc, vc, words, scale)
    # a logit off by e moves its weight by e of itself: twice that on the output
    slack = 1 + 2 * 2.0 ** -22 * abs(scale) * 2 * 64 / REL
    check(lay, out, lse, (ref, ref_lse, mag * slack))


@pytest.mark.gpu
@pytest.mark.parametrize("dtype,kv", KINDS)
@pytest.mark.parametrize("page", [0, 16])
def test_hidden_and_unused_places_may_hold_anything(dtype, kv, page):
    """NaN and infinities in cache slots past a sequence's end change nothing; in drafted tokens they reach
    the rows that attend to them, and no other."""
    lay = Layout([100, 0, 126], [6, 5, 4], 2, 64, page=page, hq=4, dtype=dtype, kv=kv, capacity=300)
    kc, vc = lay.normal(*lay.shape), lay.normal(*lay.shape)
    if kv == "e4m3":
        kc, vc = ((x.float() / s).clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)
                  for x, s in ((kc, lay.k_scale), (vc, lay.v_scale)))
    q = lay.normal(lay.rows, 4, 64)
    words = random_trees(lay, lay.gen)
    clean = run(lay, q, kc, vc, words, 0.125)
    odd = 0x7F if kv == "e4m3" else math.nan
    used = torch.zeros(kc.reshape(-1, 2, 64).shape[0], dtype=torch.bool)
    for b in range(3):
        for t in range(lay.held[b] + lay.new[b]):
            used[lay.cache_row(b, t)] = True
    for c in (kc, vc):
        c.view(-1, 2, 64)[~used] = odd
    again = run(lay, q, kc, vc, words, 0.125)
    assert torch.equal(again[0], clean[0]) and torch.equal(again[1], clean[1])
    # drafted token 2 of sequences 0 and 2
    for b in (0, 2):
        z = lay.cache_row(b, lay.held[b] + 2)
        vc.view(-1, 2, 64)[z, :, 7] = odd if kv == "e4m3" else math.inf
        vc.view(-1, 2, 64)[z, 1, 9] = odd
        kc.view(-1, 2, 64)[z, 0, 3] = odd
    got, lse, _ = run(lay, q, kc, vc, words, 0.125)
    for r in range(lay.rows):
        b = lay.row_seq[r]
        sees = b != 1 and int(words[r]) >> 2 & 1
        if not sees:
            assert torch.equal(got[r], clean[0][r]) and torch.equal(lse[r], clean[1][r])
            continue
        assert torch.isnan(lse[r, :2]).all() and torch.isnan(got[r, :2]).all()    # KV head 0: K is NaN
        assert not torch.isnan(lse[r, 2:]).any() and torch.isnan(got[r, 2:, 9]).all()
        assert (~torch.isfinite(got[r, 2:, 7])).all()
        ok = [i for i in range(64) if i not in (7, 9)]
        assert torch.equal(got[r, 2:, ok], clean[0][r, 2:, ok])


@pytest.mark.gpu
@pytest.mark.parametrize("dtype,kv", KINDS)
def test_one_drafted_token_is_a_decode_step(dtype, kv):
    """T = 1: the decode step over ctx + 1 tokens."""
    lay = Layout([500, 0, 77], [1, 1, 1], 2, 128, page=16, hq=8, dtype=dtype, kv=kv, out_dtype="f32")
    kc, vc = lay.normal(*lay.shape), lay.normal(*lay.shape)
    if kv == "e4m3":
        kc, vc = ((x.float() / s).clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)
                  for x, s in ((kc, lay.k_scale), (vc, lay.v_scale)))
    q = lay.normal(3, 8, 128)
    out, lse, _ = run(lay, q, kc, vc, None, 0.09)
    step = binding.DecodeAttention(lay.problem)
    ref, ref_lse, _ = step.run(q.cuda(), kc.cuda(), vc.cuda(), lay.table.cuda(), (lay.start + 1).cuda(), 0.09)
    mag = reference(lay, q, kc, vc, None, 0.09)[2]
    assert ((out - ref.cpu()).abs() <= 2 * REL * mag).all()
    assert torch.allclose(lse, ref_lse.cpu(), rtol=1e-5, atol=1e-5)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype,kv", KINDS)
def test_bad_lengths_and_pages_are_recorded(dtype, kv):
    lay = Layout([30, 3, 2], [2, 4, 2], 2, 64, page=16, capacity=32, hq=4, dtype=dtype, kv=kv)
    t = binding.TreeAttention(lay.problem, 8)
    kc, vc = lay.cache().cuda(), lay.cache().cuda()
    q = lay.normal(lay.rows, 4, 64).cuda()
    table, offs = lay.table.cuda(), lay.row_offsets.cuda()

    def go(ctx, offs=offs, q=q, t=t):
        out = torch.full((q.shape[0], 4, 64), 5.0, dtype=q.dtype, device="cuda")
        t.run(q, kc, vc, table, offs, torch.tensor(ctx, dtype=torch.int32, device="cuda"), None, 0.1, out=out)
        try:
            t.check_status()
        except binding.DecodeAttnError as e:
            return e.code, out
        return 0, out

    assert go([30, 3, 2])[0] == 0
    code, out = go([31, 3, 2])                     # the second drafted token has no place: left as it was
    assert code == -7 and (out[1] == 5).all() and (out[0] != 5).any() and (out[2] != 5).any()
    assert go([-1, 3, 2])[0] == -7 and go([33, 3, 2])[0] == -7 and go([2147483647, 3, 2])[0] == -7
    small = binding.TreeAttention(lay.problem, 3)
    code, out = go([30, 3, 2], t=small)            # four drafted tokens, planned for three
    assert code == -7 and (out[5] == 5).all() and (out[4] != 5).any()
    for bad in ([0, 2, 6, 800], [-4, 2, 6, 8], [0, 6, 2, 8]):
        go([30, 3, 2], offs=torch.tensor(bad, dtype=torch.int32, device="cuda"))
    for entry in (-1, lay.pool, 2147483647):
        table[1, 0] = entry
        assert go([30, 3, 2])[0] == -4
    table.copy_(lay.table)
    assert go([30, 3, 2])[0] == 0
    strict = Layout([30, 3, 2], [2, 4, 2], 2, 64, page=16, capacity=32, hq=4, dtype=dtype, kv=kv, validate=True)
    t = binding.TreeAttention(strict.problem, 8)
    t.run(q, kc, vc, table, offs, lay.start.cuda(), None, 0.1)
    with pytest.raises(binding.DecodeAttnError) as e:
        t.run(q, kc, vc, table, offs, (lay.start + 1).cuda(), None, 0.1)
    assert e.value.code == -7


@pytest.mark.gpu
@pytest.mark.parametrize("batch", [1000, 5000])
def test_many_sequences(batch):
    g = torch.Generator().manual_seed(batch)
    held = torch.randint(0, 40, (batch,), generator=g).tolist()
    new = torch.randint(0, 4, (batch,), generator=g).tolist()
    lay = Layout(held, new, 1, 64, page=16, hq=4, seed=2)
    kc, vc, q = lay.cache(), lay.cache(), lay.normal(lay.rows, 4, 64)
    words = random_trees(lay, lay.gen)
    out, lse, _ = run(lay, q, kc, vc, words, 0.125)
    check(lay, out, lse, reference(lay, q, kc, vc, words, 0.125))


@pytest.mark.gpu
@pytest.mark.parametrize("kv", ["bf16", "e4m3"])
def test_runs_repeat_exactly_and_workspaces_carry_over(kv):
    """One object, other lengths in between: the same bits again."""
    lay = Layout([2000, 10], [8, 64], 2, 128, page=16, hq=8, kv=kv, capacity=2100)
    other = Layout([5, 2032], [64, 1], 2, 128, page=16, hq=8, kv=kv, capacity=2100, spare=0)
    kc, vc, q = lay.cache(), lay.cache(), lay.normal(lay.rows, 8, 128)
    words = random_trees(lay, lay.gen)
    a = run(lay, q, kc, vc, words, 0.05)
    b = run(lay, q, kc, vc, words, 0.05, obj=a[2])
    small = min(lay.pool, other.pool)
    other.table.clamp_(max=small - 1)
    other.pool = lay.pool
    run(other, other.normal(other.rows, 8, 128), kc, vc, None, 0.05, obj=a[2])
    c = run(lay, q, kc, vc, words, 0.05, obj=a[2])
    for x in (b, c):
        assert torch.equal(a[0].view(torch.int16), x[0].view(torch.int16)) and torch.equal(a[1], x[1])


@pytest.mark.gpu
def test_captured_run_follows_lengths_and_masks():
    lay = Layout([100, 600], [6, 3], 2, 128, page=16, hq=8, capacity=1024)
    kc, vc = lay.cache().cuda(), lay.cache().cuda()
    table = torch.arange(2 * 64, dtype=torch.int32).view(2, 64) % lay.pool
    table, offs, ctx = table.cuda(), lay.row_offsets.cuda(), lay.start.cuda()
    q, words = lay.normal(lay.rows, 8, 128).cuda(), random_trees(lay, lay.gen).cuda()
    t, u = binding.TreeAttention(lay.problem, 8), binding.TreeAttention(lay.problem, 8)
    out, lse = torch.empty_like(q), torch.empty(lay.rows, 8, device="cuda")
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        t.run(q, kc, vc, table, offs, ctx, words, 0.1, out=out, out_lse=lse)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        t.run(q, kc, vc, table, offs, ctx, words, 0.1, out=out, out_lse=lse)
    for lens, split in (([1000, 3], [0, 4, 9]), ([5, 900], [1, 2, 8])):
        ctx.copy_(torch.tensor(lens, dtype=torch.int32))
        offs.copy_(torch.tensor(split, dtype=torch.int32))
        words.copy_(random_trees(lay, lay.gen))
        q.copy_(lay.normal(lay.rows, 8, 128))
        ref, ref_lse = torch.zeros_like(out), torch.zeros_like(lse)
        out.zero_()
        lse.zero_()
        u.run(q, kc, vc, table, offs, ctx, words, 0.1, out=ref, out_lse=ref_lse)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, ref) and torch.equal(lse, ref_lse)


@pytest.mark.gpu
@pytest.mark.parametrize("kv", ["bf16", "e4m3"])
def test_two_objects_on_two_streams(kv):
    lay = Layout([3000, 500], [12, 30], 2, 128, page=16, hq=8, kv=kv)
    kc, vc, q = lay.cache().cuda(), lay.cache().cuda(), lay.normal(lay.rows, 8, 128).cuda()
    place = (lay.table.cuda(), lay.row_offsets.cuda(), lay.start.cuda())
    objs = [binding.TreeAttention(lay.problem, 30) for _ in range(2)]
    ref, ref_lse = objs[0].run(q, kc, vc, *place, None, 0.1)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    outs = [[], []]
    for _ in range(20):
        for i in range(2):
            with torch.cuda.stream(streams[i]):
                outs[i].append(objs[i].run(q, kc, vc, *place, None, 0.1))
    torch.cuda.synchronize()
    for o, s in outs[0] + outs[1]:
        assert torch.equal(o.view(torch.int16), ref.view(torch.int16)) and torch.equal(s, ref_lse)


@pytest.mark.gpu
@pytest.mark.parametrize("kv", ["bf16", "e4m3"])
def test_a_speculative_step(kv):
    """Write the drafted rows (rotary by tree depth), verify the tree, move the accepted path's rows to the
    end of the context, decode the next token: against the same in float64 from the cache's own values."""
    from _rows import rotate
    hq, hkv, d = 8, 2, 64
    lay = Layout([70, 5], [6, 4], hkv, d, page=16, hq=hq, kv=kv, capacity=128, k_scale=0.0125, v_scale=0.0125,
                 out_dtype="f32")
    io = binding.KVCacheIO(lay.problem, findings=True)
    R = binding.Rope(d)
    theta = torch.tensor(R.frequencies(), dtype=torch.float64)
    kc, vc = ((torch.randn(lay.shape, generator=lay.gen) / s).clamp(-448, 448).to(torch.float8_e4m3fn)
              .view(torch.uint8) if kv == "e4m3" else lay.normal(*lay.shape) for s in (lay.k_scale, lay.v_scale))
    gk, gv = kc.cuda(), vc.cuda()
    table, offs, start = lay.table.cuda(), lay.row_offsets.cuda(), lay.start.cuda()
    words = random_trees(lay, lay.gen)
    depth = torch.tensor([bin(int(w) & ((1 << lay.new[lay.row_seq[r]]) - 1)).count("1") - 1
                          for r, w in enumerate(words)])
    pos = (depth + lay.start[torch.tensor(lay.row_seq)]).int()
    wide = lay.normal(lay.rows, hq + 2 * hkv, d)
    dev = wide.cuda()
    q = io.write(dev[:, hq:hq + hkv], dev[:, hq + hkv:], gk, gv, table, offs, start, rope=R,
                 positions=pos.cuda(), q=dev[:, :hq])
    tree = binding.TreeAttention(lay.problem, 8)
    out, lse = tree.run(q, gk, gv, table, offs, start, words.cuda(), 0.125)
    ref = reference(lay, q.cpu(), gk.cpu(), gv.cpu(), words, 0.125)
    check(lay, out.cpu(), lse.cpu(), ref)
    # the rotated q itself
    want = rotate(wide[:, :hq].double(), pos, theta, d)
    assert ((q.cpu().double() - want).abs() <= want.abs() * 2.0 ** -8 + 1e-4).all()
    # accept a path: of each sequence the last drafted token and its ancestors
    keep, r0, lens = [], 0, []
    for b, n in enumerate(lay.new):
        w = int(words[r0 + n - 1]) & ((1 << n) - 1)
        keep.append([j for j in range(n) if w >> j & 1])
        lens.append(lay.held[b] + len(keep[-1]))
        r0 += n
    k_rows, v_rows = (torch.empty(lay.rows, hkv, d, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    io.read(gk, gv, table, offs, start, k_rows, v_rows)
    at = torch.tensor([int(lay.row_offsets[b]) + j for b in range(2) for j in keep[b]], device="cuda")
    new_offs = torch.tensor([0, len(keep[0]), len(keep[0]) + len(keep[1])], dtype=torch.int32, device="cuda")
    io.write(k_rows[at], v_rows[at], gk, gv, table, new_offs, start)
    io.check_status()
    # the next decode step over the accepted tokens
    q1 = lay.normal(2, hq, d)
    got, got_lse, _ = binding.DecodeAttention(lay.problem).run(
        q1.cuda(), gk, gv, table, torch.tensor(lens, dtype=torch.int32, device="cuda"), 0.125)
    for b in range(2):
        old = lay.values(gk.cpu(), lay.k_scale), lay.values(gv.cpu(), lay.v_scale)
        rows = torch.tensor([lay.cache_row(b, t) for t in range(lens[b])])
        k, v = (c[rows].repeat_interleave(hq // hkv, 1) for c in old)
        x = torch.einsum("hd,thd->ht", q1[b].double(), k) * 0.125
        p = torch.softmax(x, -1)
        want = torch.einsum("ht,thd->hd", p, v)
        mag = torch.einsum("ht,thd->hd", p, v.abs())
        assert ((got[b].cpu().double() - want).abs() <= REL * mag).all()
        first = lay.held[b]
        src = k_rows[int(lay.row_offsets[b]) + torch.tensor(keep[b])].cpu().double()
        moved = old[0][rows[first:]]
        assert ((moved - src).abs() <= src.abs() * 2.0 ** -8).all()


@pytest.mark.gpu
@pytest.mark.parametrize("dtype,kv", KINDS)
@pytest.mark.parametrize("out_dtype", ["f32", None])
@pytest.mark.parametrize("hq,new", [(4, [3, 9, 17]), (8, [1, 11, 33]), (1, [31, 47, 1])])
def test_rows_that_fill_a_warp_in_part(dtype, kv, out_dtype, hq, new):
    """T G off the multiples of 32, over 128 columns (several a lane to store), with drafted V values that are not
    finite: some lanes of a warp store, some store and add, some do neither."""
    lay = Layout([200, 0, 640], new, 1, 128, page=16, hq=hq, dtype=dtype, kv=kv, out_dtype=out_dtype)
    kc, vc = fill_normal(lay)
    q, words = lay.normal(lay.rows, hq, 128), random_trees(lay, lay.gen, hide=0.2)
    clean, clean_lse, _ = run(lay, q, kc, vc, words, 0.09)
    check(lay, clean, clean_lse, reference(lay, q, kc, vc, words, 0.09))
    for b in range(3):
        vc.view(-1, 1, 128)[lay.cache_row(b, lay.held[b]), 0, 70] = 0x7F if kv == "e4m3" else math.nan
    got, lse, t = run(lay, q, kc, vc, words, 0.09)
    sees = torch.tensor([bool(int(w) & 1) for w in words])
    assert torch.isnan(got[sees][..., 70]).all() and torch.equal(got[~sees], clean[~sees])
    rest = [i for i in range(128) if i != 70]
    assert torch.equal(got[..., rest], clean[..., rest]) and torch.equal(lse, clean_lse)
    t.check_status()


@pytest.mark.gpu
@pytest.mark.parametrize("dtype,kv", [("bf16", "bf16"), ("f16", "f16"), ("bf16", "e4m3")])
@pytest.mark.parametrize("sms", [1, 40])
def test_runs_among_other_tensor_core_kernels(dtype, kv, sms):
    """Runs and matrix products in turn on one stream, called and captured: each kernel takes its tensor memory
    once what is ahead of it has ended (with one CTA the product follows the attention kernel itself)."""
    lay = Layout([700, 90], [8, 5], 2, 128, page=16, hq=8, dtype=dtype, kv=kv, num_sms=sms)
    kc, vc = (c.cuda() for c in fill_normal(lay))
    q = lay.normal(lay.rows, 8, 128).cuda()
    place = (lay.table.cuda(), lay.row_offsets.cuda(), lay.start.cuda())
    t = binding.TreeAttention(lay.problem, 8)
    a = torch.randint(-2, 3, (512, 512), device="cuda").to(TORCH[dtype])
    ref, ref_lse = t.run(q, kc, vc, *place, None, 0.1)
    prod = a @ a
    outs = []

    def turns(n):
        for _ in range(n):
            outs.append((a @ a, *t.run(q, kc, vc, *place, None, 0.1)))

    turns(30)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        turns(2)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        turns(4)
    for _ in range(3):
        graph.replay()
    torch.cuda.synchronize()
    for p, out, lse in outs:
        assert torch.equal(p, prod)
        assert torch.equal(out.view(torch.int16), ref.view(torch.int16)) and torch.equal(lse, ref_lse)
    t.check_status()


@pytest.mark.gpu
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("out_dtype", ["f16", "bf16"])
def test_fp8_weights_keep_their_bits_under_16_bit_results(out_dtype, d):
    """A 16-bit result over an FP8 cache is held to the fp32 bound and one rounding, as over a 16-bit cache. A few
    tokens a row, so that the roundings of weights do not average out: where terms cancel, weights of 11 bits
    (2^-11 of sum p |v|, 16 times REL) would show."""
    lay = Layout([2, 3, 1, 4, 6, 0, 9, 2], [2, 3, 5, 2, 4, 3, 1, 6], 4, d, page=8, hq=16, dtype="bf16", kv="e4m3",
                 out_dtype=out_dtype, seed=9)
    kc, vc = fill_normal(lay)
    q = lay.normal(lay.rows, 16, d)
    wide = Layout(lay.held, lay.new, 4, d, page=8, hq=16, dtype="bf16", kv="e4m3", out_dtype="f32", seed=9)
    exact, _, mag = reference(wide, q, kc, vc, None, 0.1)
    got, _, _ = run(lay, q, kc, vc, None, 0.1)
    tol = mag * REL
    tol = tol + (exact.abs() + tol) * half_step(TORCH[out_dtype]) + (2.0 ** -25 if out_dtype == "f16" else 0)
    assert ((got.double() - exact).abs() <= tol).all()
    # (the oracle with weights rounded to one f16 breaks it)
    G, worst = 4, 0.0
    k_all, v_all = lay.values(kc, lay.k_scale), lay.values(vc, lay.v_scale)
    for b, (ctx, n) in enumerate(zip(lay.held, lay.new)):
        at = torch.tensor([lay.cache_row(b, t) for t in range(ctx + n)])
        i = n - 1
        r = int(lay.row_offsets[b]) + i
        x = torch.einsum("hd,thd->ht", q[r].double(), k_all[at].repeat_interleave(G, 1)) * 0.1
        p = (x - x.amax(-1, keepdim=True)).exp()
        o = torch.einsum("ht,thd->hd", p.half().double(), v_all[at].repeat_interleave(G, 1)) / p.sum(-1)[:, None]
        o = o.to(TORCH[out_dtype]).double()
        worst = max(worst, float(((o - exact[r]).abs() / tol[r]).max()))
    assert worst > 1


@pytest.mark.gpu
@pytest.mark.parametrize("dtype,kv", KINDS)
@pytest.mark.parametrize("place", [0, 5000, 19999])
@pytest.mark.parametrize("depth", [2.25, 9.0, 12.0, 18.0])
def test_weights_far_below_a_sink(dtype, kv, place, depth):
    """One token with V = 0 holds nearly all of the weight, 20000 others lie `depth` nats below it, in one piece:
    their small weights make up the whole result. All are equal, so that roundings add up. f16 operands lose up to
    half of f16's smallest step, 2^-25, of a weight that is scaled so that the row's largest is at least 2^11:
    2^-36 of it, times sum |v|. The fp32 accumulator is rounded once for every 16 tokens and part of a weight,
    2 n / 16 times, each time by up to 2^-23 (an accumulation may cut off) of a partial sum, which with V > 0 and
    equal weights is at most sum p |v|: n / 8 * 2^-23 of it."""
    n = 20000
    lay = Layout([n - 2], [2], 1, 64, page=16, hq=2, dtype=dtype, kv=kv, k_scale=1.0, v_scale=1.0, out_dtype="f32",
                 num_sms=1)
    rows = torch.tensor([lay.cache_row(0, t) for t in range(n)])
    k, v = torch.zeros(lay.shape).view(-1, 1, 64), torch.zeros(lay.shape).view(-1, 1, 64)
    k[rows, :, 0] = -depth / 8
    v[rows] = torch.rand(n, 1, 64, generator=lay.gen) + 0.5
    k[rows[place], :, 0] = 0.0
    v[rows[place]] = 0.0
    store = torch.float8_e4m3fn if kv == "e4m3" else TORCH[dtype]
    kc, vc = (c.to(store).view(lay.shape) for c in (k, v))
    if kv == "e4m3":
        kc, vc = kc.view(torch.uint8), vc.view(torch.uint8)
    assert (k.view(-1, 64) == lay.values(kc, 1.0).view(-1, 64)).all()          # the logits are exact
    q = torch.zeros(2, 2, 64).to(TORCH[dtype])
    q[:, :, 0] = 8.0
    words = torch.tensor([3, 3], dtype=torch.int64)
    out, lse, _ = run(lay, q, kc, vc, words, 1.0)
    ref, ref_lse, mag = reference(lay, q, kc, vc, words, 1.0)
    mag = mag * (1 + n / 8 * 2.0 ** -23 / REL)
    if dtype == "f16" or kv == "e4m3":
        largest = math.exp(0.0 - float(ref_lse[0, 0]))
        mag = mag + 2.0 ** -36 / REL * largest * lay.values(vc, 1.0).abs().sum(0)
    check(lay, out, lse, (ref, ref_lse, mag))


@pytest.mark.gpu
@pytest.mark.parametrize("dtype,kv", KINDS)
@pytest.mark.parametrize("sms", [1, 40])
@pytest.mark.parametrize("first,last", [(0, 128), (128, 256), (300, 301), (0, 900)])
def test_nan_in_the_context_reaches_result_and_lse(dtype, kv, sms, first, last):
    """Keys of NaN at positions first..last - 1, a whole first tile among them: every row's out and lse are NaN,
    however the reference moves afterwards, and another sequence's are untouched."""
    lay = Layout([1000, 1000], [3, 3], 2, 64, page=16, hq=4, dtype=dtype, kv=kv, num_sms=sms)
    kc, vc = fill_normal(lay)
    q = lay.normal(lay.rows, 4, 64)
    clean = run(lay, q, kc, vc, None, 0.3)
    z = torch.tensor([lay.cache_row(0, t) for t in range(first, last)])
    kc.view(-1, 2, 64)[z] = 0x7F if kv == "e4m3" else math.nan
    out, lse, t = run(lay, q, kc, vc, None, 0.3)
    assert torch.isnan(out[:3]).all() and torch.isnan(lse[:3]).all()
    assert torch.equal(out[3:], clean[0][3:]) and torch.equal(lse[3:], clean[1][3:])
    t.check_status()


@pytest.mark.gpu
@pytest.mark.parametrize("what", ["tree", "io", "step"])
@pytest.mark.parametrize("given", [True, False])
def test_a_dropped_objects_workspace_waits_for_its_last_stream(what, given):
    """Run on a busy side stream (given, or current), then drop the object: its workspace's memory goes to nobody
    else while the run is pending."""
    lay = Layout([600, 70], [4, 3], 2, 64, page=16, hq=8)
    kc, vc, q = lay.cache().cuda(), lay.cache().cuda(), lay.normal(lay.rows, 8, 64).cuda()
    table, offs, start = lay.table.cuda(), lay.row_offsets.cuda(), lay.start.cuda()
    rows = torch.empty(lay.rows, 2, 64, dtype=torch.bfloat16, device="cuda")
    q2 = q[:2].contiguous()
    make = {"tree": lambda: binding.TreeAttention(lay.problem, 4),
            "io": lambda: binding.KVCacheIO(lay.problem, findings=True),
            "step": lambda: binding.DecodeAttention(lay.problem)}[what]

    def call(obj, stream):
        if what == "tree":
            obj.run(q, kc, vc, table, offs, start, None, 0.1, stream=stream)
        elif what == "io":
            obj.read(kc, vc, table, offs, start, rows, rows.clone(), stream=stream)
        else:
            obj.run(q2, kc, vc, table, start, 0.1, stream=stream)

    side = torch.cuda.Stream()
    call(make(), side)                       # modules loaded
    torch.cuda.synchronize()
    for _ in range(2):                       # the second object on a stream that the first has used
        obj = make()
        address, size = obj.workspace.data_ptr(), obj.workspace.numel()
        with torch.cuda.stream(side):
            torch.cuda._sleep(400_000_000)   # a fifth of a second
            if not given:
                call(obj, None)
        if given:
            call(obj, side)
        del obj
        taken = [torch.empty(size, dtype=torch.uint8, device="cuda") for _ in range(8)]
        assert not side.query() and all(t.data_ptr() != address for t in taken)
        torch.cuda.synchronize()
        del taken


# ---- waits that run out of time ---------------------------------------------------------------
def test_debug_stall_refuses_bad_arguments():
    plan, _ = binding.decode_attn_tree_plan(_prob(), 8)
    plain, _ = binding.decode_attn_tree_plan(_prob(qkv_dtype="f32", out_dtype="f32"), 8)
    for p, tensor, code in ((plan, -1, -1), (plan, 3, -1), (plain, 1, -2), (None, 0, -1)):
        with pytest.raises(binding.DecodeAttnError) as e:
            binding.decode_attn_tree_debug_stall(p, tensor)
        assert e.value.code == code
    binding.decode_attn_tree_debug_stall(plan, 2)
    binding.decode_attn_tree_debug_stall(plan, 0)
    for p in (plan, plain):
        binding.decode_attn_tree_destroy(p)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype,kv", [("bf16", "bf16"), ("f16", "f16"), ("bf16", "e4m3")])
@pytest.mark.parametrize("tensor", [1, 2])
@pytest.mark.parametrize("d,page,new", [(128, 16, [6, 5]), (64, 0, [50, 3]), (128, 0, [64, 64])])
def test_waits_that_run_out_of_time_end_the_run(dtype, kv, tensor, d, page, new):
    """CTA 0 leaves out a load: every role gives up in turn, the run ends with the timeout recorded, and the same
    object's next run is the plain one's, bit for bit."""
    lay = Layout([3000, 2500], new, 2, d, page=page, hq=8, dtype=dtype, kv=kv, num_sms=8)
    kc, vc = (c.cuda() for c in fill_normal(lay))
    q = lay.normal(lay.rows, 8, d).cuda()
    place = (lay.table.cuda() if page else None, lay.row_offsets.cuda(), lay.start.cuda())
    t = binding.TreeAttention(lay.problem, 64)
    ref, ref_lse = t.run(q, kc, vc, *place, None, 0.1)
    t.check_status()
    for _ in range(2):
        binding.decode_attn_tree_debug_stall(t.plan, tensor)
        t.run(q, kc, vc, *place, None, 0.1)
        with pytest.raises(binding.DecodeAttnError) as e:
            t.check_status()
        assert e.value.code == -6
        binding.decode_attn_tree_debug_stall(t.plan, 0)
        out, lse = t.run(q, kc, vc, *place, None, 0.1)
        t.check_status()
        assert torch.equal(out.view(torch.int16), ref.view(torch.int16)) and torch.equal(lse, ref_lse)
    lay.problem.validate = 1
    strict = binding.TreeAttention(lay.problem, 64)
    binding.decode_attn_tree_debug_stall(strict.plan, tensor)
    with pytest.raises(binding.DecodeAttnError) as e:
        strict.run(q, kc, vc, *place, None, 0.1)
    assert e.value.code == -6
