"""Pages and slots from the sequences' lengths: refusals on the CPU, results on the GPU against a model in
plain integers."""
import ctypes
import os
import shutil
import subprocess

import pytest
import torch

from decode_attention_attn_gb300 import binding, build as lib_build

A = 0x100000   # an aligned address that no refused call dereferences
HEAD = binding.POOL_HEAD


@pytest.fixture(scope="module", autouse=True)
def built():
    lib_build.build()


def _problem(batch=4, page=16, width=8, blocks=64, **kw):
    return binding.make_problem(**{**dict(
        batch=batch, num_q_heads=8, num_kv_heads=2, head_dim=64, qkv_dtype="bf16", out_dtype="bf16", paged=True,
        page_size=page, max_blocks_per_seq=width, num_physical_blocks=blocks,
        num_sms=0 if torch.cuda.is_available() else 152), **kw})


# ---- CPU: refusals --------------------------------------------------------------------------
def _code(fn, *args):
    with pytest.raises(binding.DecodeAttnError) as e:
        fn(*args)
    return e.value.code


def _set(args, kw):
    for k, v in kw.items():
        assert hasattr(args, k)
        setattr(args, k, v)
    return args


def test_calls_refuse_bad_arguments():
    plan, ws = binding.decode_attn_plan(_problem(), 0)
    checked, _ = binding.decode_attn_plan(_problem(validate=True), 0)
    contiguous, _ = binding.decode_attn_plan(_problem(paged=False, max_seq_len=64), 0)
    many, _ = binding.decode_attn_plan(_problem(batch=16385), 0)
    P = 0x1000   # (apart: 64 pages, 4 x 8 entries)

    def reserve(plan=plan, **kw):
        args = binding.da_pages_reserve_args(A, A + P, A + 2 * P, A + 3 * P, 9, A + 4 * P, A + 5 * P, A + 6 * P,
                                             A + 7 * P, ws, None)
        return _code(binding.decode_attn_pages_reserve, plan, _set(args, kw))

    def release(plan=plan, **kw):
        args = binding.da_pages_release_args(A, A + P, A + 2 * P, A + 3 * P, A + 7 * P, ws, None)
        return _code(binding.decode_attn_pages_release, plan, _set(args, kw))

    for name in ("pool", "block_table", "row_offsets", "ctx_lens"):
        assert reserve(**{name: None}) == -1, name
    for name in ("pool", "block_table", "seq_lens", "keep_lens"):
        assert release(**{name: None}) == -1, name
    assert reserve(rows=-1) == -1
    for name in ("block_table", "row_offsets", "ctx_lens", "seq_lens", "slots", "positions"):
        assert reserve(**{name: A + 8 * P + 2}) == -1, name
    assert reserve(pool=A + 8 * P + 4) == -1 and release(pool=A + 8 * P + 8) == -1
    assert release(seq_lens=A + 8 * P + 1) == -1 and release(keep_lens=A + 8 * P + 2) == -1
    # results over inputs and over one another
    assert reserve(seq_lens=A + 3 * P + 4) == -1          # ctx_lens, but not itself
    assert reserve(slots=A + 2 * P) == -1 and reserve(slots=A + 6 * P + 32) == -1
    assert reserve(positions=A + P + 4) == -1 and reserve(block_table=A + 4 * 67) == -1
    assert reserve(seq_lens=A + 3 * P, slots=A + 3 * P + 12) == -1     # in place, and a result over it
    assert release(block_table=A + 4 * 67) == -1 and release(keep_lens=A) == -1 and release(seq_lens=A + P) == -1
    for call in (reserve, release):
        assert call(workspace=A + 7 * P + 16) == -1 and call(workspace_bytes=ws - 1) == -3
        assert call(checked, workspace=None) == -1
        assert call(contiguous) == -2 and call(many) == -2
    assert _code(binding.decode_attn_pages_init, plan, 0) == -1
    assert _code(binding.decode_attn_pages_init, plan, A + 4) == -1
    assert _code(binding.decode_attn_pages_init, contiguous, A) == -2
    assert _code(binding.decode_attn_pages_init, None, A) == -1
    assert _code(binding.decode_attn_pages_reserve, None, binding.da_pages_reserve_args()) == -1
    assert _code(binding.decode_attn_pages_release, None, binding.da_pages_release_args()) == -1
    for p in (plan, checked, contiguous, many):
        binding.decode_attn_destroy(p)


def test_wrappers_refuse_bad_tensors():
    pages = binding.PageTables(_problem())
    i32 = dict(dtype=torch.int32)
    pool, table, offs, lens = (torch.zeros(n, **i32) for n in (HEAD + 64, 32, 5, 4))
    bad = torch.zeros(3, **i32)
    for args in ((bad, table, offs, lens), (pool, bad, offs, lens), (pool, table, bad, lens), (pool, table, offs, bad),
                 (pool.long(), table, offs, lens), (pool, torch.zeros(64, **i32)[::2], offs, lens)):
        with pytest.raises(ValueError):
            pages.reserve(*args, 4)
    with pytest.raises(ValueError):
        pages.reserve(pool, table, offs, lens, -1)
    for kw in (dict(slots=bad), dict(positions=bad.float()), dict(seq_lens=bad)):
        with pytest.raises(ValueError):
            pages.reserve(pool, table, offs, lens, 4, **kw)
    with pytest.raises(ValueError, match="CUDA"):
        pages.reserve(pool, table, offs, lens, 4)
    with pytest.raises(ValueError):
        pages.release(pool, table, lens, bad)
    with pytest.raises(ValueError, match="CUDA"):
        pages.release(pool, table, lens, lens)
    with pytest.raises(ValueError, match="findings"):
        pages.check_status()
    with pytest.raises(ValueError, match="no pages"):
        binding.PageTables(_problem(paged=False, max_seq_len=64))


# ---- the model ------------------------------------------------------------------------------
class Model:
    """Pools, tables and calls in plain integers."""

    def __init__(self, batch, page, width, blocks, seed=0):
        g = torch.Generator().manual_seed(seed)
        self.batch, self.page, self.width, self.blocks = batch, page, width, blocks
        self.stack = torch.randperm(blocks, generator=g).tolist()
        self.table = [[-1] * width for _ in range(batch)]
        self.lens = [0] * batch
        self.gen = g

    def tensors(self):
        pool = torch.full((HEAD + self.blocks,), 77, dtype=torch.int32)
        pool[:HEAD] = torch.tensor([len(self.stack), 0, 0, 0])
        pool[HEAD:HEAD + len(self.stack)] = torch.tensor(self.stack, dtype=torch.int32)
        return pool.cuda(), torch.tensor(self.table, dtype=torch.int32).cuda()

    def pages(self, n):
        return -(-n // self.page)

    def reserve(self, offsets, ctx, rows):
        """(seq_lens, slots, positions, missing); the tables and the stack are changed."""
        cap = self.width * self.page
        offsets = [min(max(o, 0), rows) for o in offsets]
        new = [max(b - a, 0) for a, b in zip(offsets, offsets[1:])]
        held = [min(max(c, 0), cap) for c in ctx]
        then = [max(min(max(c + t, 0), cap), h) for c, t, h in zip(ctx, new, held)]
        need = [self.pages(n) - self.pages(h) for n, h in zip(then, held)]
        slots, positions = [-1] * rows, [0] * rows
        for b in range(self.batch):
            for i in range(new[b]):
                positions[offsets[b] + i] = ctx[b] + i
        if sum(need) > len(self.stack):
            return held, slots, positions, sum(need) - len(self.stack)
        for b in range(self.batch):
            for j in range(need[b]):
                entry = self.stack.pop()
                self.table[b][self.pages(held[b]) + j] = entry if 0 <= entry < self.blocks else -1
            for i in range(new[b]):
                t = ctx[b] + i
                if 0 <= t < cap:
                    entry = self.table[b][t // self.page]
                    if 0 <= entry < self.blocks:
                        slots[offsets[b] + i] = entry * self.page + t % self.page
        return then, slots, positions, 0

    def release(self, lens, keep):
        cap = self.width * self.page
        gone = []
        for b in range(self.batch):
            n = min(max(lens[b], 0), cap)
            k = min(max(keep[b], 0), n)
            gone += [(b, j) for j in range(self.pages(k), self.pages(n))]
        if len(self.stack) + len(gone) > self.blocks:
            return
        for b, j in reversed(gone):
            entry = self.table[b][j]
            self.stack.append(entry if 0 <= entry < self.blocks else -1)
            self.table[b][j] = -1

    def check(self, pool, table, missing=0):
        head = pool[:HEAD].tolist()
        assert head == [len(self.stack), missing, 0, 0]
        assert pool[HEAD:HEAD + len(self.stack)].tolist() == self.stack
        assert table.view(self.batch, self.width).tolist() == self.table


def _offsets(new, before=0):
    out = [before]
    for n in new:
        out.append(out[-1] + n)
    return out


def _i32(v):
    return torch.tensor(v, dtype=torch.int32).cuda()


# ---- GPU ------------------------------------------------------------------------------------
@pytest.mark.gpu
@pytest.mark.parametrize("batch,page,width,new_most", [(1, 8, 3, 24), (3, 16, 40, 9), (64, 16, 20, 1), (700, 8, 12, 30),
                                                       (513, 256, 4, 700), (1025, 32, 3, 5)])
def test_steps_and_cuts(batch, page, width, new_most):
    """Steps of random lengths and cuts back, until the pool has been through several hands."""
    m = Model(batch, page, width, batch * width // 2 + width, seed=batch)
    pages = binding.PageTables(_problem(batch, page, width, m.blocks), findings=True)
    pool, table = m.tensors()
    cap = page * width
    for step in range(6):
        room = [cap - n for n in m.lens]
        new = [min(int(torch.randint(0, new_most + 1, (1,), generator=m.gen)), r) for r in room]
        before, behind = step % 3, (step * 5) % 7
        offsets = _offsets(new, before)
        rows = offsets[-1] + behind
        got = pages.reserve(pool, table, _i32(offsets), _i32(m.lens), rows)
        then, slots, positions, missing = m.reserve(offsets, m.lens, rows)
        assert [x.tolist() for x in got] == [then, slots, positions], step
        m.check(pool, table, missing)
        if not missing:
            pages.check_status()
            used = [z for z in slots if z >= 0]
            assert len(set(used)) == len(used) == sum(new)
        else:
            assert _code(pages.check_status) == -10
        m.lens = then
        keep = [int(torch.randint(0, n + 1, (1,), generator=m.gen)) if i % 3 == 0 else n for i, n in enumerate(then)]
        pages.release(pool, table, got[0], _i32(keep))
        m.release(then, keep)
        m.check(pool, table, missing)
        pages.check_status()
        m.lens = keep


@pytest.mark.gpu
def test_a_new_pool_and_a_round_trip():
    m = Model(5, 16, 8, 40)
    m.stack = list(range(39, -1, -1))
    pages = binding.PageTables(_problem(5, 16, 8, 40))
    pool = pages.new_pool()
    table = _i32(m.table)
    m.check(pool, table)
    side = torch.cuda.Stream()
    other = pages.new_pool("cuda:0", stream=side)
    side.synchronize()
    assert torch.equal(other, pool)
    offsets, lens = _offsets([17, 0, 128, 1, 16]), [0] * 5
    then, slots, _ = pages.reserve(pool, table, _i32(offsets), _i32(lens), offsets[-1])
    assert then.tolist() == [17, 0, 128, 1, 16]
    assert table.view(5, 8)[2].tolist() == [2, 3, 4, 5, 6, 7, 8, 9] and slots[:3].tolist() == [0, 1, 2]
    start = pool.clone()
    pages.release(pool, table, then, _i32(lens))
    m.check(pool, table)
    assert torch.equal(start[HEAD:], pool[HEAD:])


@pytest.mark.gpu
@pytest.mark.parametrize("short", [1, 2, 9])
def test_a_step_that_does_not_fit_takes_nothing(short):
    m = Model(6, 8, 10, 60)
    pages = binding.PageTables(_problem(6, 8, 10, 60), findings=True)
    offsets = _offsets([20, 8, 0, 31, 5, 9])
    first = m.reserve(offsets, m.lens, offsets[-1])[0]
    offsets = _offsets([9, 20, 16, 30, 3, 16])
    need = sum(m.pages(n + t) - m.pages(n) for n, t in zip(first, [9, 20, 16, 30, 3, 16]))
    m.stack = m.stack[:need - short]
    pool, table = m.tensors()
    lens = _i32(first)
    got = pages.reserve(pool, table, _i32(offsets), lens, offsets[-1], seq_lens=lens)
    assert got[0] is lens and lens.tolist() == first
    assert got[1].tolist() == [-1] * offsets[-1]
    assert got[2].tolist() == m.reserve(offsets, first, offsets[-1])[2]
    m.check(pool, table, short)
    assert _code(pages.check_status) == -10
    pages.check_status()


@pytest.mark.gpu
def test_bad_lengths_and_entries_are_recorded():
    m = Model(7, 8, 4, 64)
    pages = binding.PageTables(_problem(7, 8, 4, 64), findings=True)
    first = m.reserve(_offsets([8, 9, 30, 4, 12, 3, 20]), m.lens, 86)[0]
    # a negative length, rows past the capacity, a length past it, a bad page held, a bad page on the stack
    ctx = [first[0], -5, 30, 4, 100, 3, 20]
    new = [3, 8, 5, 2, 4, 6, 4]
    m.table[3][0] = 64
    m.stack[-1] = -9
    offsets = _offsets(new, 1)
    pool, table = m.tensors()
    got = pages.reserve(pool, table, _i32(offsets), _i32(ctx), 34)
    want = m.reserve(offsets, ctx, 34)
    assert [x.tolist() for x in got] == list(want[:3])
    m.check(pool, table)
    assert _code(pages.check_status) == -4
    # offsets that reach past the rows, and back
    offsets = [0, 3, 3, 50, 60, 60, 60, 60]
    got = pages.reserve(pool, table, _i32(offsets), _i32([0] * 7), 6)
    want = m.reserve(offsets, [0] * 7, 6)
    assert [x.tolist() for x in got] == list(want[:3])
    m.check(pool, table)
    # lengths kept past those held, negative ones, lengths past the capacity, bad entries
    m = Model(7, 8, 4, 64)
    first = m.reserve(_offsets([8, 9, 30, 4, 12, 3, 32]), m.lens, 98)[0]
    m.table[2][1] = 1000
    pool, table = m.tensors()
    pages.check_status()
    lens, keep = [8, 9, 30, -1, 12, 3, 99], [9, -3, 8, 0, 5, 3, 7]
    pages.release(pool, table, _i32(lens), _i32(keep))
    m.release(lens, keep)
    m.check(pool, table)
    assert _code(pages.check_status) == -4
    # more than the pool has room for
    before = table.clone()
    table.fill_(5)
    pages.release(pool, table, _i32([32] * 7), _i32([0] * 7))
    assert (table == 5).all() and pool[0] == len(m.stack)
    assert _code(pages.check_status) == -4
    table.copy_(before)
    m.check(pool, table)


@pytest.mark.gpu
def test_counts_out_of_range_are_clamped():
    m = Model(2, 8, 4, 10)
    pages = binding.PageTables(_problem(2, 8, 4, 10), findings=True)
    pool, table = m.tensors()
    for count, free in ((-7, 0), (1 << 30, 10)):
        pool[0] = count
        pages.reserve(pool, table, _i32([0, 0, 0]), _i32([0, 0]), 0)
        assert pool[0] == free
    pool[0] = -7
    lens, slots, _ = pages.reserve(pool, table, _i32([0, 1, 1]), _i32([0, 0]), 1)
    assert slots.tolist() == [-1] and pool[:2].tolist() == [0, 1]


@pytest.mark.gpu
def test_many_rows_and_many_sequences():
    """Several CTAs, sequences of many rows and of none, the largest batch."""
    for batch, page, new in ((16384, 16, [i % 3 for i in range(16384)]), (5, 16, [1, 700000, 0, 300007, 40000]),
                             (300, 64, [(i * i) % 4096 for i in range(300)])):
        new = torch.tensor(new)
        held = torch.arange(batch) % (2 * page + 1)
        width = int((held + new).max() + page - 1) // page
        pages_held, pages_all = (held + page - 1) // page, (held + new + page - 1) // page
        blocks = int(pages_all.sum())
        perm = torch.randperm(blocks)
        pages = binding.PageTables(_problem(batch, page, width, blocks), findings=True)
        pool = torch.zeros(HEAD + blocks, dtype=torch.int32)
        used = int(pages_held.sum())
        pool[0] = blocks - used
        pool[HEAD:HEAD + blocks - used] = perm[used:].int()
        table = torch.full((batch, width), -1, dtype=torch.int32)
        table[torch.arange(width)[None] < pages_held[:, None]] = perm[:used].int()
        pool, table = pool.cuda(), table.cuda()
        pool0, table0 = pool.clone(), table.clone()
        offsets = torch.cat([torch.zeros(1, dtype=torch.int64), new.cumsum(0)])
        rows = int(offsets[-1])
        lens, slots, positions = pages.reserve(pool, table, offsets.int().cuda(), held.int().cuda(), rows)
        b = torch.repeat_interleave(torch.arange(batch), new)
        t = held[b] + torch.arange(rows) - offsets[b]
        assert torch.equal(positions.cpu().long(), t) and torch.equal(lens.cpu().long(), held + new)
        tab = table.cpu().long()
        assert torch.equal(slots.cpu().long(), tab[b, t // page] * page + t % page)
        grid = torch.arange(width)[None]
        fresh = (grid >= pages_held[:, None]) & (grid < pages_all[:, None])
        assert torch.equal(tab[fresh], perm[used:].flip(0)) and torch.equal(tab[~fresh], table0.cpu().long()[~fresh])
        assert pool[:HEAD].tolist() == [0, 0, 0, 0]
        pages.release(pool, table, lens, held.int().cuda())
        assert torch.equal(pool, pool0) and torch.equal(table, table0)
        pages.check_status()


@pytest.mark.gpu
def test_captured_calls_follow_their_inputs_and_streams_are_taken():
    m = Model(9, 8, 30, 200)
    pages = binding.PageTables(_problem(9, 8, 30, 200))
    pool, table = m.tensors()
    offsets, lens = _i32(_offsets([4] * 9)), _i32([0] * 9)
    keep = _i32([0] * 9)
    slots, positions = torch.empty(40, dtype=torch.int32, device="cuda"), torch.empty(40, dtype=torch.int32, device="cuda")
    then = torch.empty_like(lens)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.stream(side):
        with torch.cuda.graph(graph, stream=side):
            pages.reserve(pool, table, offsets, lens, 40, seq_lens=then, slots=slots, positions=positions)
            pages.release(pool, table, then, keep)
    m.check(pool, table)
    for step in range(4):
        new = [(step * 3 + i) % 5 for i in range(9)]
        off = _offsets(new, step)
        offsets.copy_(_i32(off))
        lens.copy_(_i32(m.lens))
        want_then, want_slots, want_pos, missing = m.reserve(off, m.lens, 40)
        kept = [max(0, n - i % 4) for i, n in enumerate(want_then)]
        keep.copy_(_i32(kept))
        graph.replay()
        m.release(want_then, kept)
        assert missing == 0 and then.tolist() == want_then
        assert slots.tolist() == want_slots and positions.tolist() == want_pos
        m.check(pool, table)
        m.lens = kept
    # on a stream of the caller's
    with torch.cuda.stream(side):
        got = pages.reserve(pool, table, offsets, _i32(m.lens), 40, stream=side)
    want = m.reserve(off, m.lens, 40)
    side.synchronize()
    assert [x.tolist() for x in got] == list(want[:3])


@pytest.mark.gpu
def test_validate_returns_the_findings():
    pages = binding.PageTables(_problem(2, 8, 4, 3, validate=True))
    pool, table = pages.new_pool(), torch.full((2, 4), -1, dtype=torch.int32, device="cuda")
    lens = _i32([0, 0])
    pages.reserve(pool, table, _i32([0, 8, 16]), lens, 16)
    assert _code(pages.reserve, pool, table, _i32([0, 8, 16]), _i32([8, 8]), 16) == -10
    assert _code(pages.release, pool, table, _i32([8, 8]), _i32([0, 9])) == -7


@pytest.mark.gpu
def test_plans_of_different_batches_from_threads_at_once(tmp_path):
    """Their launches take different amounts of shared memory, of which one call must not withhold another's."""
    cxx = shutil.which("g++") or shutil.which("c++")
    if cxx is None:
        pytest.skip("no host C++ compiler")
    subprocess.run([cxx, "-std=c++17", "-O2", "-Wall", "-Werror", "-shared", "-fPIC", "-pthread",
                    os.path.join(os.path.dirname(__file__), "c_call_threads.cpp"), "-o", str(tmp_path / "threads.so")], check=True)
    call = ctypes.CDLL(str(tmp_path / "threads.so")).call_at_once
    entry = {n: ctypes.cast(getattr(binding.lib(), "decode_attn_pages_" + n), ctypes.c_void_p).value for n in ("reserve", "release")}
    for name in ("reserve", "release"):
        fns, handles, args, keep = [], [], [], []
        for batch in (16384, 8300, 6500, 9):
            pages = binding.PageTables(_problem(batch, 16, 2, 64))
            stream = torch.cuda.Stream()
            pool, table = pages.new_pool(), torch.full((batch, 2), -1, dtype=torch.int32, device="cuda")
            offsets, lens, then = (torch.zeros(batch + k, dtype=torch.int32, device="cuda") for k in (1, 0, 0))
            at = stream.cuda_stream
            a = (binding.da_pages_reserve_args(pool.data_ptr(), table.data_ptr(), offsets.data_ptr(), lens.data_ptr(), 0,
                                               then.data_ptr(), None, None, None, 0, at) if name == "reserve" else
                 binding.da_pages_release_args(pool.data_ptr(), table.data_ptr(), then.data_ptr(), lens.data_ptr(), None, 0, at))
            keep.append((pages, stream, pool, table, offsets, lens, then, a))
            fns.append(entry[name])
            handles.append(pages.plan if isinstance(pages.plan, int) else pages.plan.value)
            args.append(ctypes.addressof(a))
        torch.cuda.synchronize()
        many = ctypes.c_void_p * 4
        assert call(4, 3000, many(*fns), many(*handles), many(*args)) == 0, name
        torch.cuda.synchronize()
        assert all(k[2][0] == 64 and not k[6].any() for k in keep)


@pytest.mark.gpu
def test_offsets_that_fall_take_nothing():
    """Rows of two sequences at once: no pages leave the stack, nothing is entered, and the finding says so."""
    m = Model(5, 8, 10, 60)
    pages = binding.PageTables(_problem(5, 8, 10, 60), findings=True)
    first = m.reserve(_offsets([20, 8, 0, 31, 5]), m.lens, 64)[0]
    pool, table = m.tensors()
    for offsets, rows in (([0, 30, 10, 40, 50, 60], 60), ([0, 9, 20, 21, 22, 21], 30), ([40, 0, 1, 2, 3, 4], 64)):
        got = pages.reserve(pool, table, _i32(offsets), _i32(first), rows)
        assert [x.tolist() for x in got] == [first, [-1] * rows, [0] * rows]
        m.check(pool, table)
        assert _code(pages.check_status) == -7
    # ones that fall past the rows there are do not: no row counts there
    offsets = [0, 3, 40, 20, 30, 25]
    got = pages.reserve(pool, table, _i32(offsets), _i32(first), 12)
    want = m.reserve(offsets, first, 12)
    assert [x.tolist() for x in got] == list(want[:3]) and want[0][1] == first[1] + 9
    m.check(pool, table)
    pages.check_status()
