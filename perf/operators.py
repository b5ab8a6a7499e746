"""Cases and plain forms of the operators around a decode step: rotary positions, writing a KV
cache (with the rotary applied and the rows quantised), reading it back, and attention for a
tree of drafted tokens over the cache.

`own` chooses what run() calls: elementary torch operations, or the library."""
import math

import torch

own = False

DT = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
ES = {"f32": 4, "f16": 2, "bf16": 2, "e4m3": 1}
E4M3_MAX = 448.0
K_SCALE, V_SCALE = 0.01171875, 0.0087890625   # N(0, 1) rows: 5.25 and 3.9375 are the largest values held


# ---- the cases --------------------------------------------------------------------------------
def _rope(name, rows, heads, d, dtype, rotary, interleaved=False, scaling="none", transpose=False, gap=0, far=131072):
    return {"name": name, "op": "rope", "rows": rows, "heads": heads, "d": d, "dtype": dtype, "rotary": rotary,
            "interleaved": interleaved, "scaling": scaling, "transpose": transpose, "gap": gap, "far": far}


def _cache(name, op, batch, hq, hkv, d, dtype, kv, page, lo, hi, new_lo, new_hi, **more):
    """`batch` sequences that hold lo..hi tokens; new_lo..new_hi rows of each are written, read or drafted."""
    return {"name": name, "op": op, "batch": batch, "hq": hq, "hkv": hkv, "d": d, "dtype": dtype, "kv": kv,
            "page": page, "lo": lo, "hi": hi, "new_lo": new_lo, "new_hi": new_hi, **more}


def listed():
    return [
        # q and k heads of a decode step's fused projection rows (the v heads between rows stay as they are)
        _rope("rope_decode_64", 64, 40, 128, "bf16", 128, scaling="by_parts", gap=8),
        # the gradient of a prompt's rotary: half of each head rotated, pairs side by side
        _rope("rope_prompt_grad", 8191, 32, 128, "f16", 64, interleaved=True, scaling="linear", transpose=True),
        # one decode step of the paged batch: q and k rotated, one row of K and V appended to each sequence
        _cache("write_decode_paged_fp8", "write", 64, 32, 8, 128, "bf16", "e4m3", 16, 512, 8192, 1, 1, rotary=128),
        # a batch of prompts going into the pages
        _cache("write_prompts_paged_fp8", "write", 64, 32, 8, 128, "bf16", "e4m3", 16, 0, 0, 100, 512, rotary=128),
        # a 4K prompt into a contiguous cache of the multi-head shape, already rotated elsewhere
        _cache("write_prompt_mha_f16", "write", 1, 32, 32, 128, "f16", "f16", 0, 0, 0, 4096, 4096, rotary=0),
        # one sequence's last thousand rows, for a prefix kept elsewhere
        _cache("read_tail_f16", "read", 1, 32, 32, 128, "f16", "f16", 0, 3000, 3000, 1001, 1001),
        # the paged batch in full, back in bf16
        _cache("read_paged_fp8", "read", 64, 32, 8, 128, "bf16", "e4m3", 16, 0, 0, 512, 8192),
        # a short conversation, a small tree, 8 query heads to a KV head
        _cache("tree_short_d64", "tree", 2, 16, 2, 64, "bf16", "bf16", 8, 300, 777, 13, 13, chain=False),
        # a chain of drafts after a 4K context, one query head to a KV head
        _cache("tree_chain_mha_f16", "tree", 1, 32, 32, 128, "f16", "f16", 0, 4091, 4091, 5, 5, chain=True),
        # a tree over a 32K context
        _cache("tree_32k_bf16", "tree", 1, 32, 8, 128, "bf16", "bf16", 0, 32768, 32768, 16, 16, chain=False),
        # the paged batch, trees of different sizes
        _cache("tree_paged_bf16", "tree", 64, 32, 8, 128, "bf16", "bf16", 16, 512, 8192, 3, 12, chain=False),
        # the same batch over FP8 pages with the widest trees
        _cache("tree_paged_fp8_wide", "tree", 64, 32, 8, 128, "bf16", "e4m3", 16, 512, 8192, 64, 64, chain=False),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["rope", "write", "read", "tree", "tree"])
    dtype = rng.choice(["bf16", "bf16", "f16", "f32"])
    if op == "rope":
        d = rng.choice([64, 128])
        c = _rope("", _log(rng, 1, 8192), _log(rng, 1, 40), d, dtype, rng.choice([d, d, d // 2, d // 4]),
                  rng.random() < 0.5, rng.choice(["none", "linear", "ntk", "by_parts", "by_index"]),
                  rng.random() < 0.3, rng.choice([0, 0, 2, 8]), _log(rng, 100, 4000000))
    else:
        group, d = rng.choice([1, 2, 4, 4, 8]), rng.choice([64, 128, 128])
        hkv = rng.choice([1, 2, 3, 4, 8, 8, 16])
        while group * hkv > 64:
            hkv //= 2
        kv = "e4m3" if dtype == "bf16" and rng.random() < 0.5 else dtype
        page = rng.choice([0, 8, 16, 16, 64, 256])
        batch = _log(rng, 1, 64)
        most = max(64, 262144 // batch)   # tokens a sequence, so that a case stays below the largest listed one
        if op == "tree":
            hi = _log(rng, 1, min(32768, most if dtype != "f32" else most // 8))
            t = _log(rng, 1, 64)
            c = _cache("", "tree", batch, group * hkv, hkv, d, dtype, kv, page, rng.randint(0, hi), hi,
                       rng.randint(1, t), t, chain=rng.random() < 0.3)
        elif op == "write":
            new = _log(rng, 1, max(1, min(2048, most // 8)))
            hi = _log(rng, 1, max(1, most // 8))
            c = _cache("", "write", batch, group * hkv, hkv, d, dtype, kv, page, rng.randint(0, hi), hi,
                       rng.randint(0, new), new, rotary=rng.choice([0, d, d, d // 2]))
        else:
            hi, new = _log(rng, 1, max(1, most // 8)), _log(rng, 1, max(1, most // 8))
            c = _cache("", "read", batch, group * hkv, hkv, d, dtype, kv, page, rng.randint(0, hi), hi,
                       rng.randint(0, new), new)
    del c["name"]
    return c


# ---- what a caller has in hand ----------------------------------------------------------------
def _lens(case, g):
    """Tokens held and rows to come of each sequence: a case's own, in an order of `g`'s, so that the sizes of
    pools and outputs are the case's."""
    own_g = torch.Generator().manual_seed(4)
    held, new = (torch.randint(case[lo], case[hi] + 1, (case["batch"],), generator=own_g)
                 for lo, hi in (("lo", "hi"), ("new_lo", "new_hi")))
    new[0] = max(1, int(new[0]))
    order = torch.randperm(case["batch"], generator=g)
    return held[order], new[order]


def _scaling(case):
    """The rotary of a case as the library's constructor takes it."""
    kind = case.get("scaling", "none")
    r = {"head_dim": case["d"], "rotary_dim": case["rotary"], "interleaved": case.get("interleaved", False),
         "base": 500000.0 if kind == "by_parts" else 10000.0, "scaling": kind}
    if kind != "none":
        r["factor"] = 8.0
    if kind in ("by_parts", "by_index"):
        r["original_max_position"] = 8192
        r["low"], r["high"] = (1.0, 4.0) if kind == "by_parts" else (1.0, 32.0)
    if kind == "by_index":
        r["attn_factor"] = 1.2079441541679836
    return r


def _frequencies(r):
    """theta_i of each rotated pair, in 64 bits."""
    n, base = r["rotary_dim"], r["base"]
    i = torch.arange(n // 2, dtype=torch.float64)
    kind, s = r["scaling"], r.get("factor", 1.0)
    if kind == "ntk":
        base = base * s ** (n / (n - 2)) if n > 2 else base
    theta = base ** (-2.0 * i / n)
    if kind == "linear":
        theta = theta / s
    elif kind == "by_parts":   # turns over the original context
        turns = r["original_max_position"] * theta / (2 * math.pi)
        keep = ((turns - r["low"]) / (r["high"] - r["low"])).clamp(0, 1)
        theta = theta / s * (1 - keep) + theta * keep
    elif kind == "by_index":
        at = lambda turns: n * math.log(r["original_max_position"] / (turns * 2 * math.pi)) / (2 * math.log(base))
        first, last = max(math.floor(at(r["high"])), 0), min(math.ceil(at(r["low"])), n - 1)
        keep = 1 - ((i - first) / max(last - first, 0.001)).clamp(0, 1)
        theta = theta / s * (1 - keep) + theta * keep
    return theta


def prepare(case, seed):
    dev = torch.device("cuda")
    g = torch.Generator().manual_seed(seed)                  # lengths, tables, trees
    gd = torch.Generator(device=dev).manual_seed(seed)       # values
    d, dt = case["d"], DT[case["dtype"]]

    def normal(*shape, dtype=dt):
        return torch.randn(shape, generator=gd, device=dev, dtype=torch.float32).to(dtype)

    s = {"case": case}
    if case["op"] == "rope":
        wide = normal(case["rows"], case["heads"] + case["gap"], d)
        s["x"] = wide[:, :case["heads"]]
        s["positions"] = torch.randint(0, case["far"], (case["rows"],), generator=g).int().to(dev)
        s["rope"] = _scaling(case)
        s["theta"] = _frequencies(s["rope"]).to(dev)
        s["out"] = torch.empty((case["rows"], case["heads"], d), dtype=dt, device=dev)
        if own:
            from decode_attention_attn_gb300 import binding
            s["handle"] = binding.Rope(**s["rope"])
        return s

    B, hkv, page = case["batch"], case["hkv"], case["page"]
    held, new = _lens(case, g)
    total = held + new
    s["rows"], s["most"], s["most_new"] = int(new.sum()), max(1, int(total.max())), max(1, int(new.max()))
    s["start"] = held.int().to(dev)
    s["row_offsets"] = torch.cat([torch.zeros(1, dtype=torch.int64), new.cumsum(0)]).int().to(dev)
    if page:
        pages = (total + page - 1) // page
        s["blocks"] = max(1, int(pages.sum()))
        perm = torch.randperm(s["blocks"], generator=g)
        table = torch.full((B, max(1, int(pages.max()))), -1, dtype=torch.int64)
        used = torch.arange(table.shape[1])[None, :] < pages[:, None]
        table[used] = perm[:int(pages.sum())]
        s["table"] = table.int().to(dev)
        shape = (s["blocks"], page, hkv, d)
    else:
        s["table"] = None
        shape = (B, s["most"], hkv, d)
    fp8 = case["kv"] == "e4m3"
    s["k_scale"], s["v_scale"] = (K_SCALE, V_SCALE) if fp8 else (1.0, 1.0)
    for name, scale in (("k_cache", s["k_scale"]), ("v_cache", s["v_scale"])):
        if fp8:
            x = (normal(*shape, dtype=torch.float32) / scale).clamp(-E4M3_MAX, E4M3_MAX).to(torch.float8_e4m3fn)
        else:
            x = normal(*shape)
        s[name] = x
    rows = s["rows"]
    s["scale"] = 1.0 / math.sqrt(d)
    if case["op"] == "write":
        # q, k and v are parts of one projection's rows
        wide = normal(rows, case["hq"] + 2 * hkv, d)
        s["q"], s["k"], s["v"] = wide[:, :case["hq"]], wide[:, case["hq"]:case["hq"] + hkv], wide[:, case["hq"] + hkv:]
        if case["rotary"]:
            s["rope"] = _scaling(case)
            s["theta"] = _frequencies(s["rope"]).to(dev)
            s["q_out"] = torch.empty((rows, case["hq"], d), dtype=dt, device=dev)
    elif case["op"] == "read":
        s["k_out"], s["v_out"] = (torch.empty((rows, hkv, d), dtype=dt, device=dev) for _ in range(2))
    else:
        s["q"] = normal(rows, case["hq"], d)
        s["out"] = torch.empty_like(s["q"])
        s["lse"] = torch.empty((rows, case["hq"]), dtype=torch.float32, device=dev)
        s["mask"] = None if case["chain"] else _trees(new, g).to(dev)
    if own:
        from decode_attention_attn_gb300 import binding
        problem = binding.make_problem(
            batch=B, num_q_heads=case["hq"], num_kv_heads=hkv, head_dim=d, qkv_dtype=case["dtype"],
            out_dtype=case["dtype"], paged=bool(page), page_size=page or 16,
            max_blocks_per_seq=s["table"].shape[1] if page else 0, num_physical_blocks=s["blocks"] if page else 0,
            max_seq_len=0 if page else s["most"], kv_dtype=case["kv"], k_scale=s["k_scale"], v_scale=s["v_scale"])
        if case["op"] == "tree":
            s["handle"] = binding.TreeAttention(problem, max_tree=s["most_new"])
        else:
            s["handle"] = binding.KVCacheIO(problem)
            if "rope" in s:
                s["rope_handle"] = binding.Rope(**s["rope"])
    return s


def _trees(new, g):
    """A random tree for each sequence: node i hangs below an earlier node (or the context), and attends to
    its ancestors and itself. One 64-bit word a row, bit j for node j."""
    words = []
    for n in new.tolist():
        of = []
        for i in range(n):
            p = int(torch.randint(-1, i, (1,), generator=g)) if i else -1
            of.append((of[p] if p >= 0 else 0) | 1 << i)
        words += [w - (1 << 64) if w >= 1 << 63 else w for w in of]
    return torch.tensor(words, dtype=torch.int64)


# ---- the plain forms --------------------------------------------------------------------------
def _rotate(x, positions, theta, r, transpose=False):
    """x [rows, heads, d] in 32 bits, rotated; the angles of far positions in 64."""
    n, m = r["rotary_dim"], r.get("attn_factor", 1.0)
    angle = positions.double()[:, None] * theta
    cos, sin = (angle.cos() * m).float()[:, None], (angle.sin() * m).float()[:, None]
    if transpose:
        sin = -sin
    part, rest = x[..., :n], x[..., n:]
    if r["interleaved"]:
        a, b = part[..., 0::2], part[..., 1::2]
        y = torch.stack([a * cos - b * sin, b * cos + a * sin], -1).flatten(-2)
    else:
        a, b = part[..., :n // 2], part[..., n // 2:]
        y = torch.cat([a * cos - b * sin, b * cos + a * sin], -1)
    return torch.cat([y, rest], -1)


def _places(s):
    """Of every row: its sequence, its cache position, and the cache row that holds it."""
    case, offsets = s["case"], s["row_offsets"].long()
    row = torch.arange(s["rows"], device=offsets.device)
    b = torch.searchsorted(offsets, row, right=True) - 1
    t = s["start"].long()[b] + row - offsets[b]
    if case["page"]:
        z = s["table"].long()[b, t // case["page"]] * case["page"] + t % case["page"]
    else:
        z = b * s["most"] + t
    return b, t, z


def _tree_mask(s):
    """[B, most_new, most] truth values: which cache positions each drafted row attends to."""
    offsets, start = s["row_offsets"].long(), s["start"].long()
    dev = offsets.device
    new = offsets[1:] - offsets[:-1]
    i = torch.arange(s["most_new"], device=dev)
    there = i[None, :] < new[:, None]
    j = torch.arange(s["most"], device=dev)[None, :] - start[:, None]        # draft index of each position
    if s["mask"] is None:
        seen = j[:, None, :] <= i[None, :, None]
    else:
        row = (offsets[:-1, None] + i).clamp(max=s["rows"] - 1)
        bits = s["mask"][row]
        seen = (bits[:, :, None] >> j.clamp(0, 63)[:, None, :]) & 1 == 1
        seen = seen | (j < 0)[:, None, :]
    return seen & (j < new[:, None])[:, None, :] & there[:, :, None]


def _own(s):
    case, h = s["case"], s["handle"]
    if case["op"] == "rope":
        h.apply(s["x"], s["positions"], out=s["out"], transpose=case["transpose"])
        return s["out"]
    if case["op"] == "write":
        if case["rotary"]:
            h.write(s["k"], s["v"], s["k_cache"], s["v_cache"], s["table"], s["row_offsets"], s["start"],
                    rope=s["rope_handle"], q=s["q"], q_out=s["q_out"])
            return s["k_cache"], s["v_cache"], s["q_out"]
        h.write(s["k"], s["v"], s["k_cache"], s["v_cache"], s["table"], s["row_offsets"], s["start"])
        return s["k_cache"], s["v_cache"]
    if case["op"] == "read":
        return h.read(s["k_cache"], s["v_cache"], s["table"], s["row_offsets"], s["start"], s["k_out"], s["v_out"])
    return h.run(s["q"], s["k_cache"], s["v_cache"], s["table"], s["row_offsets"], s["start"], s["mask"],
                 s["scale"], out=s["out"], out_lse=s["lse"])


def run(s):
    if own:
        return _own(s)
    case = s["case"]
    dt, d = DT[case["dtype"]], case["d"]
    if case["op"] == "rope":
        return _rotate(s["x"].float(), s["positions"], s["theta"], s["rope"], case["transpose"]).to(dt)
    hkv, fp8 = case["hkv"], case["kv"] == "e4m3"
    k_rows, v_rows = s["k_cache"].view(-1, hkv, d), s["v_cache"].view(-1, hkv, d)
    if case["op"] == "write":
        b, t, z = _places(s)
        k, v = s["k"].float(), s["v"].float()
        if case["rotary"]:
            k = _rotate(k, t, s["theta"], s["rope"])
        if fp8:
            k = (k / s["k_scale"]).clamp(-E4M3_MAX, E4M3_MAX).to(torch.float8_e4m3fn)
            v = (v / s["v_scale"]).clamp(-E4M3_MAX, E4M3_MAX).to(torch.float8_e4m3fn)
            k_rows.view(torch.uint8)[z] = k.view(torch.uint8)
            v_rows.view(torch.uint8)[z] = v.view(torch.uint8)
        else:
            k_rows[z] = k.to(dt)
            v_rows[z] = v.to(dt)
        if case["rotary"]:
            return s["k_cache"], s["v_cache"], _rotate(s["q"].float(), t, s["theta"], s["rope"]).to(dt)
        return s["k_cache"], s["v_cache"]
    if case["op"] == "read":
        z = _places(s)[2]
        if fp8:
            return ((k_rows.view(torch.uint8)[z].view(torch.float8_e4m3fn).float() * s["k_scale"]).to(dt),
                    (v_rows.view(torch.uint8)[z].view(torch.float8_e4m3fn).float() * s["v_scale"]).to(dt))
        return k_rows[z], v_rows[z]
    # tree: every sequence padded to the longest, a masked softmax over it
    B, hq, page, most, new = case["batch"], case["hq"], case["page"], s["most"], s["most_new"]
    t = torch.arange(most, device=s["q"].device)
    if page:
        z = s["table"].long().clamp(min=0)[:, t // page] * page + t % page
    else:
        z = torch.arange(B, device=t.device)[:, None] * most + t
    if fp8:
        k = k_rows.view(torch.uint8)[z].view(torch.float8_e4m3fn).float() * s["k_scale"]
        v = v_rows.view(torch.uint8)[z].view(torch.float8_e4m3fn).float() * s["v_scale"]
    else:
        k, v = k_rows[z].float(), v_rows[z].float()
    seen = _tree_mask(s)
    offsets = s["row_offsets"].long()
    row = (offsets[:-1, None] + torch.arange(new, device=t.device)).clamp(max=s["rows"] - 1)
    q = s["q"][row].float().view(B, new, hkv, hq // hkv, d).permute(0, 2, 1, 3, 4).reshape(B, hkv, -1, d)
    x = (q @ k.permute(0, 2, 3, 1) * s["scale"]).view(B, hkv, new, hq // hkv, most)
    x = x.masked_fill(~seen[:, None, :, None, :], -math.inf)
    top = x.amax(-1, keepdim=True)
    p = (x - top.clamp(min=-1e30)).exp()
    total = p.sum(-1, keepdim=True)
    o = p.view(B, hkv, -1, most) @ v.permute(0, 2, 1, 3)
    o = o.view(B, hkv, new, hq // hkv, d) / total.clamp(min=1e-30)
    lse = (total.log() + top).squeeze(-1)
    o, lse = o.permute(0, 2, 1, 3, 4).reshape(B, new, hq, d), lse.permute(0, 2, 1, 3).reshape(B, new, hq)
    b, at, _ = _places(s)
    i = at - s["start"].long()[b]
    return o[b, i].to(dt), lse[b, i]


# ---- what a pass cannot do without ------------------------------------------------------------
def work(case):
    d, es = case["d"], ES[case["dtype"]]
    if case["op"] == "rope":
        n = case["rows"] * case["heads"]
        return {"bytes": 2 * n * d * es + 4 * case["rows"], "flops": 3 * n * case["rotary"]}
    B, hq, hkv, kes = case["batch"], case["hq"], case["hkv"], ES[case["kv"]]
    held, new = (case["lo"] + case["hi"]) / 2 * B, (case["new_lo"] + case["new_hi"]) / 2 * B
    small = 8 * B + (4 * B * ((held + new) / B / case["page"]) if case["page"] else 0)
    if case["op"] == "write":
        q = 2 * new * hq * d * es if case["rotary"] else 0
        return {"bytes": 2 * new * hkv * d * (es + kes) + q + small,
                "flops": 3 * new * (hq + hkv) * case["rotary"] + 2 * new * hkv * d}
    if case["op"] == "read":
        return {"bytes": 2 * new * hkv * d * (es + kes) + small, "flops": 2 * new * hkv * d}
    rows = new
    return {"bytes": 2 * (held + new) * hkv * d * kes + 2 * rows * hq * d * es + 4 * rows * hq + small
            + (0 if case["chain"] else 8 * rows), "flops": 4 * rows * hq * d * (held + new) / B}


# ---- the definitions in 64 bits ---------------------------------------------------------------
def exact(case, seed):
    s = prepare(case, seed)
    d = case["d"]

    def turn(x, pos, r, sign=1.0):
        """Each pair as a complex number times m e^(i theta t)."""
        n = r["rotary_dim"]
        w = torch.polar(torch.full((n // 2,), float(r.get("attn_factor", 1.0)), dtype=torch.float64, device=x.device)
                        .expand(len(pos), -1).contiguous(), sign * pos.double()[:, None] * s["theta"])[:, None]
        y = x.double().clone()
        if r["interleaved"]:
            c = torch.complex(y[..., 0:n:2].contiguous(), y[..., 1:n:2].contiguous()) * w
            y[..., 0:n:2], y[..., 1:n:2] = c.real, c.imag
        else:
            c = torch.complex(y[..., :n // 2].contiguous(), y[..., n // 2:n].contiguous()) * w
            y[..., :n // 2], y[..., n // 2:n] = c.real, c.imag
        return y

    if case["op"] == "rope":
        return turn(s["x"], s["positions"], s["rope"], -1.0 if case["transpose"] else 1.0)
    offsets, start = s["row_offsets"].tolist(), s["start"].tolist()

    def rows_of(b, t0, t1):
        """The cache rows of positions t0..t1 of sequence b."""
        t = torch.arange(t0, t1)
        if not case["page"]:
            return b * s["most"] + t
        return s["table"][b].long().cpu()[t // case["page"]] * case["page"] + t % case["page"]

    flat = {n: s[n].view(-1, case["hkv"], d) for n in ("k_cache", "v_cache")}
    if case["op"] == "write":
        at = torch.cat([rows_of(b, start[b], start[b] + offsets[b + 1] - offsets[b]) for b in range(case["batch"])])
        pos = torch.cat([torch.arange(start[b], start[b] + offsets[b + 1] - offsets[b]) for b in range(case["batch"])])
        at, pos = at.to(s["k"].device), pos.to(s["k"].device)
        k, v = s["k"].double(), s["v"].double()
        if case["rotary"]:
            k = turn(k, pos, s["rope"])
        if case["kv"] == "e4m3":
            k, v = ((x / y).clamp(-E4M3_MAX, E4M3_MAX) for x, y in ((k, s["k_scale"]), (v, s["v_scale"])))
        full = [flat[n].double() for n in ("k_cache", "v_cache")]
        full[0][at], full[1][at] = k, v
        full = tuple(x.view(s["k_cache"].shape) for x in full)
        return full + (turn(s["q"], pos, s["rope"]),) if case["rotary"] else full
    if case["op"] == "read":
        at = torch.cat([rows_of(b, start[b], start[b] + offsets[b + 1] - offsets[b]) for b in range(case["batch"])])
        at = at.to(s["k_cache"].device)
        if case["kv"] == "e4m3":
            k, v = (flat[n].view(torch.uint8)[at].view(torch.float8_e4m3fn).double() for n in ("k_cache", "v_cache"))
            return k * s["k_scale"], v * s["v_scale"]
        return flat["k_cache"][at].double(), flat["v_cache"][at].double()
    if work(case)["flops"] > 4e12:
        return None
    dev, group = s["q"].device, case["hq"] // case["hkv"]
    out = torch.zeros(s["q"].shape, dtype=torch.float64, device=dev)
    lse = torch.full(s["lse"].shape, -math.inf, dtype=torch.float64, device=dev)
    for b in range(case["batch"]):
        n = offsets[b + 1] - offsets[b]
        if not n:
            continue
        at = rows_of(b, 0, start[b] + n).to(dev)
        if case["kv"] == "e4m3":
            k, v = (flat[c].view(torch.uint8)[at].view(torch.float8_e4m3fn).double() * y
                    for c, y in (("k_cache", s["k_scale"]), ("v_cache", s["v_scale"])))
        else:
            k, v = flat["k_cache"][at].double(), flat["v_cache"][at].double()
        hidden = torch.zeros(n, start[b] + n, dtype=torch.bool)
        for i in range(n):
            word = int(s["mask"][offsets[b] + i]) if s["mask"] is not None else (1 << i + 1) - 1
            for j in range(n):
                hidden[i, start[b] + j] = not word >> j & 1
        hidden = hidden.to(dev)
        q = s["q"][offsets[b]:offsets[b + 1]].double()
        for h in range(case["hkv"]):
            part = q[:, h * group:(h + 1) * group]
            x = torch.einsum("igd,td->igt", part, k[:, h]) * s["scale"]
            x = x.masked_fill(hidden[:, None, :], -math.inf)
            norm = torch.logsumexp(x, -1)
            out[offsets[b]:offsets[b + 1], h * group:(h + 1) * group] = torch.einsum("igt,td->igd", (x - norm[..., None]).exp(), v[:, h])
            lse[offsets[b]:offsets[b + 1], h * group:(h + 1) * group] = norm
    return out, lse
