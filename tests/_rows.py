"""Helpers of the tests of the operators around a step: ragged row layouts over a cache, and plain
float64 forms written apart from the library."""
import math

import torch

from decode_attention_attn_gb300 import binding

TORCH = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}


class Layout:
    """A cache of `batch` sequences of up to `capacity` tokens, `held` tokens in each, and `new` rows of
    each, with `before` / `behind` padding rows that belong to no sequence."""

    def __init__(self, held, new, hkv, d, page=0, capacity=None, before=0, behind=0, spare=2, seed=0,
                 hq=None, dtype="bf16", kv=None, k_scale=0.0125, v_scale=0.0075, out_dtype=None,
                 validate=False, num_sms=0):
        g = torch.Generator().manual_seed(seed)
        self.held, self.new, self.hkv, self.d, self.page = list(held), list(new), hkv, d, page
        self.hq, self.dtype, self.kv = hq or hkv, dtype, kv or dtype
        self.batch, self.rows = len(self.held), before + sum(self.new) + behind
        total = [h + n for h, n in zip(self.held, self.new)]
        cap = max(1, capacity or max(total))
        offs = [before]
        for n in self.new:
            offs.append(offs[-1] + n)
        self.row_offsets = torch.tensor(offs, dtype=torch.int32)
        self.start = torch.tensor(self.held, dtype=torch.int32)
        # of every row: sequence (-1: none) and position
        self.row_seq = [-1] * self.rows
        self.row_pos = [0] * self.rows
        for b, n in enumerate(self.new):
            for i in range(n):
                self.row_seq[offs[b] + i], self.row_pos[offs[b] + i] = b, self.held[b] + i
        if page:
            blocks = (cap + page - 1) // page
            self.capacity = blocks * page
            need = [(t + page - 1) // page for t in total]
            self.pool = sum(need) + spare
            perm = torch.randperm(self.pool, generator=g)
            self.table = torch.full((self.batch, blocks), -1, dtype=torch.int32)
            at = 0
            for b, n in enumerate(need):
                self.table[b, :n] = perm[at:at + n].int()
                at += n
            self.shape = (self.pool, page, hkv, d)
        else:
            self.capacity, self.table, self.shape = cap, None, (self.batch, cap, hkv, d)
        fp8 = self.kv == "e4m3"
        self.k_scale, self.v_scale = (k_scale, v_scale) if fp8 else (1.0, 1.0)
        self.problem = binding.make_problem(
            batch=self.batch, num_q_heads=self.hq, num_kv_heads=hkv, head_dim=d, qkv_dtype=dtype,
            out_dtype=out_dtype or dtype, paged=bool(page), page_size=page or 16,
            max_blocks_per_seq=self.table.shape[1] if page else 0,
            num_physical_blocks=self.pool if page else 0, max_seq_len=0 if page else cap,
            kv_dtype=self.kv, k_scale=self.k_scale, v_scale=self.v_scale, validate=validate,
            num_sms=num_sms or (0 if torch.cuda.is_available() else 152))
        self.gen = g

    def normal(self, *shape):
        return torch.randn(shape, generator=self.gen).to(TORCH[self.dtype])

    def cache(self):
        """A cache of random values (random codes without NaN for FP8)."""
        if self.kv == "e4m3":
            c = torch.randint(0, 256, self.shape, generator=self.gen, dtype=torch.uint8)
            return torch.where((c & 0x7F) == 0x7F, torch.zeros_like(c), c)
        return self.normal(*self.shape)

    def cache_row(self, b, t):
        """Row of the flat [tokens, H_kv, d] view that holds token t of sequence b, or None."""
        if not 0 <= t < self.capacity:
            return None
        if not self.page:
            return b * self.capacity + t
        entry = int(self.table[b, t // self.page])
        return entry * self.page + t % self.page if 0 <= entry < self.pool else None

    def values(self, cache, scale):
        """The float64 values of a cache, flat."""
        flat = cache.reshape(-1, self.hkv, self.d)
        if self.kv == "e4m3":
            return flat.view(torch.float8_e4m3fn).double() * scale
        return flat.double()


def frequencies(rotary, base=10000.0, scaling="none", factor=1.0, original=0.0, low=1.0, high=32.0):
    n = rotary
    if scaling == "ntk" and n > 2:
        base = base * factor ** (n / (n - 2))
    out = []
    at = lambda turns: n * math.log(original / (turns * 2 * math.pi)) / (2 * math.log(base))
    for i in range(n // 2):
        theta, keep = base ** (-2.0 * i / n), 1.0
        if scaling == "linear":
            keep = 0.0
        elif scaling == "by_parts":
            keep = min(max((original * theta / (2 * math.pi) - low) / (high - low), 0.0), 1.0)
        elif scaling == "by_index":
            a, b = max(math.floor(at(high)), 0), min(math.ceil(at(low)), n - 1)
            keep = 1 - min(max((i - a) / max(b - a, 0.001), 0.0), 1.0)
        out.append(theta / factor * (1 - keep) + theta * keep)
    return torch.tensor(out, dtype=torch.float64)


def rotate(x, positions, theta, rotary, interleaved=False, m=1.0, transpose=False):
    """x [rows, heads, d] float64, the pair as a 2 x 2 matrix at each position."""
    a = (positions.double()[:, None] * theta)[:, None, :]
    c, s = m * a.cos(), m * a.sin() * (-1 if transpose else 1)
    y = x.clone()
    i = torch.arange(rotary // 2)
    p, q = (2 * i, 2 * i + 1) if interleaved else (i, i + rotary // 2)
    y[..., p] = c * x[..., p] - s * x[..., q]
    y[..., q] = s * x[..., p] + c * x[..., q]
    return y


def rotate_bound(x, positions, theta, rotary, interleaved=False, m=1.0):
    """What the fp32 rotation may be off by, before the rounding to the output's type. The angle is
    exact but for its last conversion (2^-25 of at most pi) and the bits below 2^-32 turns; cos and sin
    of it are within 2 ulp (2^-23 of at most 1): 4e-7 in all, on each of |a| and |b|; the products and
    the sum add at most three roundings of 2^-24. The reference's own angle is off by 2^-52 of it."""
    err = 4e-7 + 3 * 2.0 ** -24 + (positions.double().abs()[:, None] * theta)[:, None, :] * 2.0 ** -51
    i = torch.arange(rotary // 2)
    p, q = (2 * i, 2 * i + 1) if interleaved else (i, i + rotary // 2)
    both = (x[..., p].abs() + x[..., q].abs()) * err * abs(m)
    out = torch.zeros_like(x)
    out[..., p], out[..., q] = both, both
    return out


def half_step(t):
    """Largest rounding of a value of type t, relative."""
    return torch.finfo(t).eps / 2
