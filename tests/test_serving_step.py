"""A step of a serving loop through the operators one after another: pages from the lengths, norm with the residual,
projection beside the requests' adapters, norms of q and k heads, rotary and write, attention over what was written,
and the pages given back."""
import pytest
import torch

from _rows import frequencies, half_step, rotate
from decode_attention_attn_gb300 import binding, build as lib_build

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def built():
    lib_build.build()


HQ, HKV, D, N, PAGE, RANK = 8, 2, 64, 256, 16, 16
OUTS = [HQ * D, HKV * D, HKV * D]


class Model:
    """One layer's weights, and the operators over a cache of `blocks` pages."""

    def __init__(self, batch, kv, blocks, width):
        g = torch.Generator().manual_seed(7)
        bf = lambda *s, gain=1.0: (gain * torch.randn(*s, generator=g)).bfloat16().cuda()
        self.norm_w, self.qk_w = 1 + 0.2 * bf(N), 1 + 0.2 * bf(D)
        self.w = bf(sum(OUTS), N, gain=N ** -0.5)
        self.a, self.b = bf(3, 3 * RANK, N, gain=N ** -0.5), bf(3, sum(OUTS), RANK, gain=0.3)
        self.scales = torch.tensor([0.5, 1.0, 2.0], device="cuda")
        self.problem = binding.make_problem(
            batch=batch, num_q_heads=HQ, num_kv_heads=HKV, head_dim=D, qkv_dtype="bf16", out_dtype="f32", paged=True,
            page_size=PAGE, max_blocks_per_seq=width, num_physical_blocks=blocks, kv_dtype=kv, k_scale=2.0 ** -5,
            v_scale=2.0 ** -5)
        self.pages = binding.PageTables(self.problem, findings=True)
        self.norm, self.qk_norm = binding.RMSNorm(N, eps=1e-5), binding.RMSNorm(D, eps=1e-6)
        self.adapters = binding.Adapters(N, OUTS, RANK, "bf16")
        self.rope, self.io = binding.Rope(D), binding.KVCacheIO(self.problem, findings=True)
        self.tree = binding.TreeAttention(self.problem, 64)
        self.decode = binding.DecodeAttention(self.problem)
        dt = torch.uint8 if kv == "e4m3" else torch.bfloat16
        self.kc, self.vc = (torch.zeros(blocks, PAGE, HKV, D, dtype=dt, device="cuda") for _ in range(2))
        self.pool = self.pages.new_pool()
        self.table = torch.full((batch, width), -1, dtype=torch.int32, device="cuda")
        self.lens = torch.zeros(batch, dtype=torch.int32, device="cuda")

    def step(self, x, residual, offsets, ids, chain=True):
        """(attention's output, lse, q as it was used, rows' slots); the cache holds the step's rows then."""
        lens, slots, positions = self.pages.reserve(self.pool, self.table, offsets, self.lens, x.shape[0])
        h, residual = self.norm.apply(x, self.norm_w, residual=residual)
        y = h @ self.w.t()
        self.adapters.apply(h, y, self.a, self.b, self.scales, offsets, ids, out=y)
        rows = y.view(-1, HQ + 2 * HKV, D)
        q, k, v = rows[:, :HQ], rows[:, HQ:HQ + HKV], rows[:, HQ + HKV:]
        self.qk_norm.apply(q, self.qk_w, out=q)
        self.qk_norm.apply(k, self.qk_w, out=k)
        q = self.io.write(k, v, self.kc, self.vc, self.table, offsets, self.lens, rope=self.rope, q=q)
        out, lse = self.tree.run(q, self.kc, self.vc, self.table, offsets, self.lens, None, D ** -0.5)
        return out, lse, q, slots, positions, lens, rows, residual


@pytest.mark.parametrize("kv", ["bf16", "e4m3"])
def test_a_run_of_steps(kv):
    """Prompts, a decode step, drafts that are turned down in part, a sequence that ends: every step against 64-bit
    forms from its own inputs, and the cache's rows at the slots."""
    batch, width = 4, 12
    m = Model(batch, kv, 40, width)
    theta = frequencies(D)
    g = torch.Generator().manual_seed(3)
    history = [[] for _ in range(batch)]              # slots of each sequence's tokens
    steps = [([40, 1, 64, 17], [0, -1, 2, 1]), ([1, 1, 1, 1], [0, -1, 2, 1]), ([5, 0, 7, 3], [0, -1, 2, 2])]
    for new, ids in steps:
        offsets = torch.tensor([0] + torch.tensor(new).cumsum(0).tolist(), dtype=torch.int32).cuda()
        rows = sum(new)
        x, res = (torch.randn(rows, N, generator=g).bfloat16().cuda() for _ in range(2))
        held = m.lens.tolist()
        id_t = torch.tensor(ids, dtype=torch.int32).cuda()
        out, lse, q, slots, positions, lens, qkv, res_out = m.step(x, res, offsets, id_t)
        m.pages.check_status(), m.io.check_status(), m.tree.check_status()
        assert lens.tolist() == [h + n for h, n in zip(held, new)]
        of = [b for b, n in enumerate(new) for _ in range(n)]
        pos = [held[b] + i for b, n in enumerate(new) for i in range(n)]
        assert positions.tolist() == pos
        for r, z in enumerate(slots.tolist()):
            history[of[r]].append(z)
        assert all(len(set(h)) == len(h) for h in history)
        # the rows that went in: norm, projection with adapters, q/k norms, rotary (bf16 between the operators)
        u = (x.float() + res.float()).bfloat16()
        assert torch.equal(u, res_out)
        hd = u.double() / (u.double().square().mean(-1, keepdim=True) + 1e-5).sqrt() * m.norm_w.double()
        y = hd @ m.w.double().t()
        for r in range(rows):
            a = ids[of[r]]
            if a < 0:
                continue
            low = hd[r] @ m.a[a].double().t()
            y[r] += float(m.scales[a]) * torch.cat([m.b[a, s:e].double() @ low[i * RANK:(i + 1) * RANK] for i, (s, e) in
                                                    enumerate(((0, 512), (512, 640), (640, 768)))])
        y = y.view(rows, HQ + 2 * HKV, D)
        unit = lambda t: t / (t.square().mean(-1, keepdim=True) + 1e-6).sqrt() * m.qk_w.double()
        turn = lambda t: rotate(t.cpu(), torch.tensor(pos), theta, D)
        want_q, want_k, want_v = turn(unit(y[:, :HQ])), turn(unit(y[:, HQ:HQ + HKV])), y[:, HQ + HKV:].cpu()
        # Roundings to bf16 on the way: h (and with it the products), y twice, q after its norm and its rotary. The
        # products' are of h's and w's terms: half a step of the magnitudes' root sum of squares, 2^-8 |h|_rms, which
        # the unit norms keep at about 1: six half steps of values up to 6 bound each element generously.
        tol = 6 * half_step(torch.bfloat16) * 6
        assert (q.cpu().double() - want_q).abs().max() < tol
        at = slots.long()
        values = lambda c: c.view(-1, HKV, D)[at].view(torch.float8_e4m3fn).double().cpu() * 2.0 ** -5 if kv == "e4m3" else \
            c.view(-1, HKV, D)[at].double().cpu()
        step = 2.0 ** -4 * 6 if kv == "e4m3" else 0.0
        assert (values(m.kc) - want_k).abs().max() < tol + step
        assert (values(m.vc) - want_v).abs().max() < tol + step * 2
        # attention from the cache's own values at the slots the pages gave
        flat = lambda c: c.view(-1, HKV, D).view(torch.float8_e4m3fn).double() * 2.0 ** -5 if kv == "e4m3" else \
            c.view(-1, HKV, D).double()
        kd, vd = flat(m.kc), flat(m.vc)
        for r in range(rows):
            z = torch.tensor(history[of[r]][:pos[r] + 1]).cuda()
            k, v = (t[z].repeat_interleave(HQ // HKV, 1) for t in (kd, vd))
            lg = torch.einsum("hd,thd->ht", q[r].double(), k) * D ** -0.5
            p = torch.softmax(lg, -1)
            err = (out[r].double() - torch.einsum("ht,thd->hd", p, v)).abs()
            assert (err <= 2.0 ** -15 * torch.einsum("ht,thd->hd", p, v.abs()) + 1e-7).all(), r
            assert (lse[r].double() - torch.logsumexp(lg, -1)).abs().max() < 1e-4
        # a decode step over the grown tables sees the same lengths
        last = offsets[1:].long() - 1
        if min(new) > 0:
            alone, alone_lse, _ = m.decode.run(q[last].contiguous(), m.kc, m.vc, m.table, lens, D ** -0.5)
            assert (alone_lse - lse[last]).abs().max() < 1e-4
            assert (alone - out[last]).abs().max() < 2e-3 * vd.abs().max()
        # some drafts are turned down, the last sequence ends
        keep = [n - (n - h) // 2 if len(new) and max(new) < 10 else n for h, n in zip(held, lens.tolist())]
        if new == steps[-1][0]:
            keep[3] = 0
        m.pages.release(m.pool, m.table, lens, torch.tensor(keep, dtype=torch.int32).cuda())
        m.pages.check_status()
        m.lens = torch.tensor(keep, dtype=torch.int32).cuda()
        for b in range(batch):
            del history[b][keep[b]:]
        used = sum(-(-n // PAGE) for n in keep)
        assert m.pool[0] == 40 - used and int((m.table >= 0).sum()) == used


def test_a_captured_step_follows_its_lengths():
    """Norm, adapters, pages, write and attention in one graph, replayed as sequences grow over their pages."""
    batch = 3
    m, eager = Model(batch, "bf16", 30, 8), Model(batch, "bf16", 30, 8)
    offsets = torch.arange(batch + 1, dtype=torch.int32).cuda()
    ids = torch.tensor([1, -1, 2], dtype=torch.int32).cuda()
    x, res = (torch.zeros(batch, N, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    m.step(x, res, offsets, ids)                     # everything is loaded
    m.pool.copy_(eager.pool), m.table.copy_(eager.table), m.kc.zero_(), m.vc.zero_()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out, lse, _, slots, _, lens, _, _ = m.step(x, res, offsets, ids)
        m.lens.copy_(lens)
    m.lens.zero_()
    g = torch.Generator().manual_seed(1)
    for i in range(35):
        x.copy_(torch.randn(batch, N, generator=g)), res.copy_(torch.randn(batch, N, generator=g))
        graph.replay()
        want = eager.step(x, res, offsets, ids)
        eager.lens = want[5]
        assert torch.equal(out, want[0]) and torch.equal(lse, want[1]) and torch.equal(slots, want[3]), i
        assert torch.equal(m.lens, eager.lens) and torch.equal(m.pool, eager.pool)
    assert m.lens.tolist() == [35] * 3
