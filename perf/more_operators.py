"""Cases and plain forms of the operators that a serving loop of many requests runs beside attention over
a paged cache: pages and slots from the requests' lengths, root-mean-square norms (of hidden rows with the
residual's addition, of q and k heads; with an output in 8 bits), and the requests' low-rank adapters beside
a shared projection.

`own` chooses what run() calls: elementary torch operations, or the library."""
import math

import torch

own = False

DT = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
ES = {"f32": 4, "f16": 2, "bf16": 2}
E4M3_MAX = 448.0
HEAD = 4            # words of a pool before its stack of free pages: [0] how many are free, [1] how many were missing


# ---- the cases --------------------------------------------------------------------------------
def _pages(name, batch, page, lo, hi, new_lo, new_hi):
    """`batch` sequences that hold lo..hi tokens get new_lo..new_hi more each, and give them back."""
    return {"name": name, "op": "pages", "batch": batch, "page": page, "lo": lo, "hi": hi, "new_lo": new_lo, "new_hi": new_hi}


def _norm(name, rows, heads, n, dtype, residual, quant, wide_weight=False, offset=0.0, gap=0):
    """quant: "none", or an output in 8 bits with a scale given for the "tensor", or one found for each "row" or
    for each "32", "64" or "128" elements."""
    return {"name": name, "op": "norm", "rows": rows, "heads": heads, "n": n, "dtype": dtype, "residual": residual,
            "quant": quant, "wide_weight": wide_weight, "offset": offset, "gap": gap}


def _adapters(name, batch, new_lo, new_hi, width, outs, rank, adapters, dtype, spread="any", bare=0.0):
    """new_lo..new_hi rows of each of `batch` requests, `width` wide, beside a projection to `outs` (widths of its
    parts). spread: requests choose their adapter alike ("any"), mostly the first ones ("few"), or each has
    its own ("each"); a share `bare` of them has none."""
    return {"name": name, "op": "adapters", "batch": batch, "new_lo": new_lo, "new_hi": new_hi, "width": width,
            "outs": outs, "rank": rank, "adapters": adapters, "dtype": dtype, "spread": spread, "bare": bare}


def listed():
    return [
        # one decode step of the paged batch: a page is taken where a sequence crosses into it
        _pages("pages_decode_64", 64, 16, 512, 8192, 1, 1),
        # drafted trees of many sequences, all of them turned down
        _pages("pages_drafts_1000", 1000, 16, 512, 8192, 3, 12),
        # a batch of prompts is let in, and let go at its end
        _pages("pages_prompts_256", 256, 16, 0, 0, 1, 8192),
        # a decode step's hidden rows: residual added, 8-bit rows for the next projection
        _norm("norm_decode_row8", 64, 1, 4096, "bf16", True, "row"),
        # q and k heads of a prompt's fused projection rows, before the rotary (the v heads between rows stay)
        _norm("norm_heads_f16", 8191, 40, 128, "f16", False, "none", gap=8),
        # a large batch of prompts, 8-bit with a scale for every 128 elements
        _norm("norm_prompts_group8", 8192, 1, 8192, "bf16", True, "128"),
        # an odd width in fp32, scale known from a calibration
        _norm("norm_odd_f32", 1001, 1, 5119, "f32", True, "tensor", offset=1.0),
        # one request decodes: q, k and v of 32/8 heads of 128
        _adapters("adapters_one", 1, 1, 1, 4096, "4096,1024,1024", 16, 8, "bf16"),
        # a decode step in which each request has an adapter of its own
        _adapters("adapters_decode_each", 64, 1, 1, 4096, "4096,1024,1024", 16, 64, "bf16", "each"),
        # drafted tokens of many requests, most with one of a few adapters, some without
        _adapters("adapters_drafts_few", 200, 1, 8, 4096, "4096,4096,4096", 32, 32, "f16", "few", 0.2),
        # a batch of prompts, the largest rank
        _adapters("adapters_prompts", 16, 100, 1024, 4096, "4096,1024,1024", 64, 8, "bf16"),
        # odd widths in fp32
        _adapters("adapters_odd_f32", 5, 1, 300, 1001, "999,77", 8, 4, "f32"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["pages", "norm", "norm", "adapters", "adapters"])
    dtype = rng.choice(["bf16", "bf16", "f16", "f32"])
    if op == "pages":
        batch = _log(rng, 1, 4096)
        most = (1 << 20) // batch     # new tokens a sequence, so that a case stays below the largest listed one
        new, hi = _log(rng, 1, max(1, min(8192, most))), _log(rng, 1, max(1, min(32768, 4 * most)))
        c = _pages("", batch, rng.choice([8, 16, 16, 32, 64, 256]), rng.randint(0, hi), hi, rng.randint(0, new), new)
    elif op == "norm":
        heads = rng.choice([1, 1, _log(rng, 2, 64)])
        n = rng.choice([64, 128, 256]) if heads > 1 else _log(rng, 64, 16384)
        n = n if heads > 1 or rng.random() < 0.2 else max(64, n // 64 * 64)
        rows = _log(rng, 1, max(1, min(16384, (1 << 26) // (n * heads * ES[dtype] // 2))))
        c = _norm("", rows, heads, n, dtype, rng.random() < 0.6, rng.choice(["none", "none", "tensor", "row", "row", "32", "64", "128"]),
                  rng.random() < 0.3, rng.choice([0.0, 0.0, 1.0]), rng.choice([0, 0, 1, 8]) if heads > 1 else 0)
    else:
        odd = rng.random() < 0.2
        size = lambda lo, hi: _log(rng, lo, hi) if odd else max(lo, _log(rng, lo, hi) // 64 * 64)
        width, outs = size(64, 8192), [size(64, 8192 // k) for k in [rng.choice([1, 1, 2, 3, 4])] for _ in range(k)]
        rank = rng.choice([8, 16, 16, 32, 64, 128])
        rank = min(rank, 64) if len(outs) * rank > 256 else rank
        one = rank * (len(outs) * width + sum(outs))                     # numbers of one adapter
        batch = _log(rng, 1, max(1, min(256, (1 << 27) // one)))
        adapters = _log(rng, 1, max(1, min(128, (1 << 27) // one)))
        if dtype == "f32":      # (whose products cost several times as much)
            batch = max(1, batch // 4)
        new = _log(rng, 1, max(1, min(1024, (8192 if dtype != "f32" else 1024) // batch)))
        c = _adapters("", batch, rng.randint(0, new), new, width, ",".join(map(str, outs)), rank, adapters, dtype,
                      rng.choice(["any", "few"]), rng.choice([0.0, 0.3]))
    del c["name"]
    return c


# ---- what a caller has in hand ----------------------------------------------------------------
def _offsets(new):
    return torch.cat([torch.zeros(1, dtype=torch.int64), new.cumsum(0)])


def _lens(case, g):
    """Tokens held (where there are any) and rows to come of each sequence: a case's own, in an order of `g`'s, so
    that the sizes of pools and outputs are the case's."""
    own_g = torch.Generator().manual_seed(4)
    held, new = (torch.randint(case.get(lo, 0), case.get(hi, 0) + 1, (case["batch"],), generator=own_g)
                 for lo, hi in (("lo", "hi"), ("new_lo", "new_hi")))
    new[0] = max(1, int(new[0]))
    order = torch.randperm(case["batch"], generator=g)
    return held[order], new[order]


def prepare(case, seed):
    dev = torch.device("cuda")
    g = torch.Generator().manual_seed(seed)                  # lengths, tables, choices
    gd = torch.Generator(device=dev).manual_seed(seed)       # values

    def normal(*shape):
        return torch.randn(shape, generator=gd, device=dev, dtype=torch.float32)

    s = {"case": case}
    if case["op"] == "pages":
        B, page = case["batch"], case["page"]
        held, new = _lens(case, g)
        pages_held, pages_all = (held + page - 1) // page, (held + new + page - 1) // page
        s["rows"], s["blocks"] = int(new.sum()), int(pages_all.sum()) + 7
        width = max(1, int(pages_all.max()))
        perm = torch.randperm(s["blocks"], generator=g).int()
        table = torch.full((B, width), -1, dtype=torch.int32)
        used = int(pages_held.sum())
        table[torch.arange(width)[None, :] < pages_held[:, None]] = perm[:used]
        pool = torch.zeros(HEAD + s["blocks"], dtype=torch.int32)
        pool[0] = s["blocks"] - used
        pool[HEAD:HEAD + s["blocks"] - used] = perm[used:]
        s["table"], s["pool"] = table.to(dev), pool.to(dev)
        s["held"], s["row_offsets"] = held.int().to(dev), _offsets(new).int().to(dev)
        if own:
            from decode_attention_attn_gb300 import binding
            s["handle"] = binding.PageTables(binding.make_problem(
                batch=B, num_q_heads=32, num_kv_heads=8, head_dim=128, qkv_dtype="bf16", out_dtype="bf16", paged=True,
                page_size=page, max_blocks_per_seq=width, num_physical_blocks=s["blocks"]))
        return s

    dt = DT[case["dtype"]]
    if case["op"] == "norm":
        rows, heads, n = case["rows"], case["heads"], case["n"]
        gains = (0.5 * normal(n)).exp()
        gains[torch.randint(0, n, (max(1, n // 500),), generator=g).to(dev)] *= 20     # a few channels stand out
        wide = (normal(rows, heads + case["gap"], n) * gains).to(dt)
        s["x"] = wide[:, :heads]
        s["residual"] = (3 * normal(rows, heads, n)).to(dt) if case["residual"] else None
        s["weight"] = (1.0 - case["offset"] + 0.3 * normal(n)).to(torch.float32 if case["wide_weight"] else dt)
        q = case["quant"]
        s["scale"] = torch.full((1,), 0.0234375, device=dev) if q == "tensor" else None
        if own:
            from decode_attention_attn_gb300 import binding
            s["handle"] = binding.RMSNorm(n, eps=1e-5, weight_offset=case["offset"])
        return s

    B, outs, rank, n = case["batch"], _outs(case), case["rank"], case["adapters"]
    _, new = _lens(case, g)
    s["rows"], s["most_new"] = int(new.sum()), int(new.max())
    s["row_offsets"] = _offsets(new).int().to(dev)
    if case["spread"] == "each":
        ids = torch.randperm(max(n, B), generator=g)[:B] % n
    elif case["spread"] == "few":
        ids = (n * torch.rand(B, generator=g) ** 4).long().clamp(max=n - 1)
    else:
        ids = torch.randint(0, n, (B,), generator=g)
    ids[torch.rand(B, generator=g) < case["bare"]] = -1
    s["ids"] = ids.int().to(dev)
    s["x"] = normal(s["rows"], case["width"]).to(dt)
    s["y"] = normal(s["rows"], sum(outs)).to(dt)
    s["a"] = (normal(n, len(outs) * rank, case["width"]) / math.sqrt(case["width"])).to(dt)
    s["b"] = (0.5 * normal(n, sum(outs), rank) / math.sqrt(rank)).to(dt)
    s["scales"] = (0.5 + 1.5 * torch.rand(n, generator=g)).to(dev)
    s["out"] = torch.empty_like(s["y"])
    if own:
        from decode_attention_attn_gb300 import binding
        s["handle"] = binding.Adapters(case["width"], outs, rank, case["dtype"])
    return s


def _outs(case):
    return [int(w) for w in case["outs"].split(",")]


# ---- the plain forms --------------------------------------------------------------------------
def _own(s):
    case, h = s["case"], s["handle"]
    if case["op"] == "pages":
        # the step's pages and slots; then the sequences are cut back to what they held
        lens, slots, positions = h.reserve(s["pool"], s["table"], s["row_offsets"], s["held"], s["rows"])
        h.release(s["pool"], s["table"], lens, s["held"])
        return lens, slots, positions, s["table"], s["pool"]
    if case["op"] == "norm":
        q = case["quant"]
        if q == "none":
            return h.apply(s["x"], s["weight"], residual=s["residual"])
        if q == "tensor":
            codes, _, total = h.quantise(s["x"], s["weight"], residual=s["residual"], scaling="tensor", scales=s["scale"])
            return codes, total
        return h.quantise(s["x"], s["weight"], residual=s["residual"], scaling="row" if q == "row" else "group",
                          group=128 if q == "row" else int(q))
    return h.apply(s["x"], s["y"], s["a"], s["b"], s["scales"], s["row_offsets"], s["ids"], out=s["out"])


def run(s):
    if own:
        return _own(s)
    return {"pages": _plain_pages, "norm": _plain_norm, "adapters": _plain_adapters}[s["case"]["op"]](s)


def _plain_pages(s):
    B, page = s["case"]["batch"], s["case"]["page"]
    table, pool, dev = s["table"], s["pool"], s["table"].device
    held, offsets, width = s["held"].long(), s["row_offsets"].long(), s["table"].shape[1]
    # the step's new pages come off the end of the stack, sequence by sequence
    lens = held + offsets[1:] - offsets[:-1]
    pages_held, pages_all = (held + page - 1) // page, (lens + page - 1) // page
    before = (pages_all - pages_held).cumsum(0) - (pages_all - pages_held)
    free = pool[0].long()
    row = torch.arange(s["rows"], device=dev)
    b = torch.searchsorted(offsets[1:], row, right=True)
    t = held[b] + row - offsets[b]
    p = t // page
    fresh = p >= pages_held[b]
    taken = pool[(HEAD + free - 1 - before[b] - (p - pages_held[b])).clamp(min=HEAD)]
    entry = torch.where(fresh, taken, table.view(-1)[b * width + p])
    slots = entry * page + (t % page).int()
    grown = torch.cat([table.view(-1), table.new_zeros(1)])       # the last place takes what is not written
    grown.scatter_(0, torch.where(fresh, b * width + p, B * width), entry)
    # the release: pages past what was held go back, the last first
    grid = torch.arange(width, device=dev)[None, :]
    gone = ((grid >= pages_held[:, None]) & (grid < pages_all[:, None])).view(-1)
    order = gone.long().cumsum(0)
    total = order[-1]
    stack = torch.cat([pool, pool.new_zeros(1)])
    stack.scatter_(0, torch.where(gone, HEAD + free - total + (total - order), len(pool)), grown[:-1])
    pool.copy_(stack[:-1])
    table.copy_(torch.where(gone, grown.new_full((), -1), grown[:-1]).view(B, width))
    return lens.int(), slots.int(), t.int(), table, pool


def _plain_norm(s):
    case, q, dt = s["case"], s["case"]["quant"], DT[s["case"]["dtype"]]
    x, total = s["x"].float(), None
    if case["residual"]:
        total = (x + s["residual"].float()).to(dt)      # what the next block adds to; the norm is of these
        x = total.float()
    r = torch.rsqrt(x.square().mean(-1, keepdim=True) + 1e-5)
    y = x * r * (s["weight"].float() + case["offset"])
    if q == "none":
        return y.to(dt) if total is None else (y.to(dt), total)
    if q == "tensor":
        codes = (y / s["scale"]).clamp(-E4M3_MAX, E4M3_MAX).to(torch.float8_e4m3fn)
        return codes, total
    group = case["n"] if q == "row" else int(q)
    groups = -(-case["n"] // group)
    y = torch.nn.functional.pad(y, (0, groups * group - case["n"])).unflatten(-1, (groups, group))
    scale = (y.abs().amax(-1) / E4M3_MAX).clamp(min=2.0 ** -126)
    codes = (y / scale[..., None]).clamp(-E4M3_MAX, E4M3_MAX).to(torch.float8_e4m3fn).flatten(-2).view(torch.uint8)
    codes = codes[..., :case["n"]].contiguous().view(torch.float8_e4m3fn)
    return codes, scale.squeeze(-1) if q == "row" else scale, total


def _plain_adapters(s):
    case, outs, rank = s["case"], _outs(s["case"]), s["case"]["rank"]
    offsets, ids, new = s["row_offsets"].long(), s["ids"].long(), s["most_new"]
    which = ids.clamp(min=0)
    i = torch.arange(new, device=ids.device)
    padded = (offsets[:-1, None] + i).clamp(max=s["rows"] - 1)            # every request padded to the longest
    low = torch.bmm(s["x"][padded].float(), s["a"][which].float().mT)
    b = s["b"][which].float()
    ends = [sum(outs[:k + 1]) for k in range(len(outs))]
    delta = torch.cat([torch.bmm(low[..., k * rank:(k + 1) * rank], b[:, e - w:e].mT)
                       for k, (e, w) in enumerate(zip(ends, outs))], -1)
    delta = delta * (s["scales"][which] * (ids >= 0))[:, None, None]
    row = torch.arange(s["rows"], device=ids.device)
    of = torch.searchsorted(offsets[1:], row, right=True)
    return (s["y"].float() + delta[of, row - offsets[of]]).to(DT[case["dtype"]])


# ---- what a pass cannot do without ------------------------------------------------------------
def work(case):
    if case["op"] == "pages":
        B, page = case["batch"], case["page"]
        rows = B * (case["new_lo"] + case["new_hi"]) / 2
        taken = rows / page
        # lengths and offsets in, lengths, slots and positions out; an entry of the stack and the table for each
        # page taken, both again (and the emptied entry) for each given back; the pages that rows go on in
        return {"bytes": 4 * (5 * B + 2 * rows + 5 * taken), "flops": 4 * rows}
    if case["op"] == "norm":
        n, es = case["rows"] * case["heads"] * case["n"], ES[case["dtype"]]
        q = case["quant"]
        scales = {"none": 0, "tensor": 0, "row": case["rows"] * case["heads"]}.get(q)
        if scales is None:
            scales = case["rows"] * case["heads"] * -(-case["n"] // int(q))
        return {"bytes": n * (es + (2 * es if case["residual"] else 0) + (es if q == "none" else 1)) + 4 * scales
                + case["n"] * (4 if case["wide_weight"] else es), "flops": 5 * n}
    B, outs, rank, es = case["batch"], _outs(case), case["rank"], ES[case["dtype"]]
    rows = B * (case["new_lo"] + case["new_hi"]) / 2
    asked = B * (1 - case["bare"])
    n = case["adapters"]
    if case["spread"] == "each":
        used = min(n, asked)
    elif case["spread"] == "few":       # adapter i is chosen with probability ((i + 1) / n)^(1/4) - (i / n)^(1/4)
        p = [((i + 1) / n) ** 0.25 - (i / n) ** 0.25 for i in range(n)]
        used = sum(1 - (1 - v) ** asked for v in p)
    else:
        used = n * (1 - (1 - 1 / n) ** asked)
    one = rank * (len(outs) * case["width"] + sum(outs))
    return {"bytes": es * (rows * (1 - case["bare"]) * case["width"] + 2 * rows * sum(outs) + used * one) + 8 * B,
            "flops": 2 * rows * (1 - case["bare"]) * one}


# ---- the definitions in 64 bits ---------------------------------------------------------------
def exact(case, seed):
    if case["op"] == "pages":
        return None                     # whole numbers
    s = prepare(case, seed)
    if case["op"] == "norm":
        h, total = s["x"].double(), None
        if s["residual"] is not None:
            total = h + s["residual"].double()
            h = total.to(DT[case["dtype"]]).double()
        size = (torch.einsum("rhn,rhn->rh", h, h) / case["n"] + 1e-5).sqrt()
        y = h * (s["weight"].double() + case["offset"]) / size[..., None]
        q = case["quant"]
        if q == "none":
            return y if total is None else (y, total)
        if q == "tensor":
            return (y / s["scale"].double()).clamp(-E4M3_MAX, E4M3_MAX), total
        parts = y.split(case["n"] if q == "row" else int(q), -1)
        scales = [p.abs().amax(-1).clamp(min=2.0 ** -126 * E4M3_MAX) / E4M3_MAX for p in parts]
        codes = torch.cat([p / c[..., None] for p, c in zip(parts, scales)], -1)
        return codes, scales[0] if q == "row" else torch.stack(scales, -1), total
    outs, rank, offsets = _outs(case), case["rank"], s["row_offsets"].tolist()
    result = s["y"].double()
    for b, a in enumerate(s["ids"].tolist()):
        lo, hi = offsets[b], offsets[b + 1]
        if a < 0 or lo == hi:
            continue
        x, at = s["x"][lo:hi].double(), 0
        for k, w in enumerate(outs):
            down, up = s["a"][a, k * rank:(k + 1) * rank].double(), s["b"][a, at:at + w].double()
            result[lo:hi, at:at + w] += float(s["scales"][a]) * (x @ down.T @ up.T)
            at += w
    return result
