"""Plain float64 forms of the narrow-cache and eviction operators, for their tests.

Caches are described by their definition in include/mimoattn.h: `slots_of` gives the float64
values that a block's slots stand for, whatever its format; `pages_of` a sequence's slots."""
import math

import numpy as np
import torch

import global_attention_attn_b200 as M

BF16, E4M3, INT4 = M.MIMO_DTYPE_BF16, M.MIMO_DTYPE_FP8_E4M3, M.MIMO_DTYPE_INT4
SCALE = 1.0 / math.sqrt(192.0)


def _int4_bytes(dims, key):
    """(byte of a row of codes, shift within it) of every dim."""
    d = np.arange(dims)
    w = d // 8
    word = (w % 4) * 6 + w // 4 if key else w
    return word * 4 + (d % 8) // 2, 4 * (d % 2)


def int4_values(block, slots, dims):
    """float64 [..., slots, dims] of 4-bit blocks [..., slots * bytes] (uint8 tensor)."""
    key = dims == 192
    byte, shift = _int4_bytes(dims, key)
    n = slots * dims // 2
    codes = block[..., :n].reshape(*block.shape[:-1], slots, dims // 2)
    c = (codes[..., torch.from_numpy(byte).to(block.device)].int() >> torch.from_numpy(shift).to(block.device)) & 15
    s = block[..., n:].contiguous().view(torch.half).reshape(*block.shape[:-1], slots, dims // 32).double()
    return (c.double() - 8) * s.repeat_interleave(32, -1)


def int4_block(codes, scales):
    """4-bit blocks from codes [..., slots, dims] (0..15) and fp16 scales [..., slots, dims / 32]."""
    dims = codes.shape[-1]
    byte, shift = _int4_bytes(dims, dims == 192)
    rows = torch.zeros(*codes.shape[:-1], dims // 2, dtype=torch.uint8, device=codes.device)
    for d in range(dims):
        rows[..., byte[d]] |= (codes[..., d] << int(shift[d])).to(torch.uint8)
    return torch.cat([rows.flatten(-2), scales.half().contiguous().view(torch.uint8).flatten(-2)], -1)


def int4_quantise(x):
    """(codes 1..15, fp16 scales) of float32 rows [..., dims], by the append's rule."""
    g = x.unflatten(-1, (-1, 32))
    s = (g.abs().amax(-1) / 7).half()
    n = torch.where(s[..., None] > 0, torch.round(g / s.float()[..., None]).clamp(-7, 7), torch.zeros_like(g))
    return (n + 8).flatten(-2).to(torch.uint8), s


def slots_of(cache, fmt, dims, dequant=None):
    """float64 [blocks, Hkv, slots, dims] of a whole cache."""
    if fmt == INT4:
        slots = cache.shape[-1] // (dims // 2 + dims // 16)
        return int4_values(cache, slots, dims)
    x = cache.transpose(1, 2)
    if fmt == E4M3:
        return x.contiguous().view(torch.float8_e4m3fn).double() * dequant.double()[None, :, None, None]
    if dims == 192:
        return torch.cat([x[..., :64].contiguous().view(torch.half).double(), x[..., 64:].double()], -1)
    return x.double()


def pages_of(values, table_row, n):
    """float64 [Hkv, n, dims]: the first n slots of a sequence."""
    pages = table_row[: -(-n // 128)].long()
    return values[pages].transpose(0, 1).flatten(1, 2)[:, :n]


def rotate(x, pos, base):
    """float64 rows [n, heads, 192] rotated at pos [n]."""
    x = x.double()
    a = pos.double()[:, None] * base ** (-torch.arange(32, dtype=torch.float64, device=x.device) / 32)
    c, s = a.cos()[:, None], a.sin()[:, None]
    u, v = x[..., :32], x[..., 32:64]
    return torch.cat([u * c - v * s, v * c + u * s, x[..., 64:]], -1)


class Row:
    """One sequence's attention: keys / values float64 [Hkv, n, dims] at slot positions `at`."""

    def __init__(self, q, k, v, at, me, base, *, pos=None, window=0, sink=None, v_scale=M.V_SCALE, p_step=2.0 ** -10):
        """q [q_len, 64, 192]; me [q_len] slot of each query row; pos [q_len] its rotary position; p_step:
        what a weight's rounding is off by (fp16 twice: 2 x 2^-11; bf16: 2^-8)."""
        self.p_step = p_step
        hkv = k.shape[0]
        qr = rotate(q, me if pos is None else pos, base).view(len(me), hkv, 64 // hkv, 192)
        z = torch.einsum("ihgd,htd->ihgt", qr, k) * SCALE
        see = at[None] <= me[:, None]
        if window:
            see &= at[None] > me[:, None] - window
        z = torch.where(see[:, None, None], z, torch.full_like(z, -math.inf))
        lse = torch.logsumexp(z, -1)
        if sink is not None:
            lse = torch.logaddexp(lse, sink.double().view(1, hkv, -1))
        self.p = torch.exp(z - lse[..., None])
        self.lse = lse.flatten(1)
        if v is not None:
            self.out = torch.einsum("ihgt,htd->ihgd", self.p, v).flatten(1, 2) * v_scale
            self.mean_abs = torch.einsum("ihgt,htd->ihgd", self.p, v.abs()).flatten(1, 2) * abs(v_scale)
            self.grid = torch.einsum("ihgt,htd->ihgd", self.p, v.abs().amax(-1, keepdim=True).expand_as(v)).flatten(1, 2)
        # what rounding the rotated dims of q to fp16 (a relative 2^-11) can move a logit by
        self.dz = float((torch.einsum("ihgd,htd->ihgt", qr[..., :64].abs(), k[..., :64].abs()) * SCALE).max()) * 2.0 ** -11

    def check(self, out, lse, what=""):
        """bf16 output within half a step of its own plus what the kernel's roundings can do: a
        logit error moves every weight by it, twice (numerator and sum); a weight is rounded to
        a narrow type once or twice (p_step); the fp32 sums of weight * code, codes up to 15 against a
        largest value of 7, keep 2^-14 of the grid's size."""
        err = (out.double() - self.out).abs()
        tol = 2.0 ** -8 * self.out.abs() + (2 * self.dz + self.p_step) * self.mean_abs + 2.0 ** -14 * self.grid
        worst = float((err / tol).max())
        assert torch.isfinite(out).all() and worst <= 1, f"{what}: output off by {worst:.3g} of its bound"
        if lse is not None:
            e = float((lse.double() - self.lse).abs().max())
            assert e <= self.dz + 1e-5, f"{what}: lse off by {e:.3g} (bound {self.dz + 1e-5:.3g})"


def table_of(lens, r, spare=2, device="cuda"):
    """Block table over a shuffled pool (ids behind a sequence's pages are -1) and the pool's size."""
    n = [-(-int(x) // 128) for x in lens]
    pool = r.permutation(sum(n) + spare).astype(np.int32)
    t = np.full((len(lens), max(max(n), 1)), -1, np.int32)
    at = 0
    for s, k in enumerate(n):
        t[s, :k] = pool[at:at + k]
        at += k
    return torch.from_numpy(t).to(device), len(pool)


def i32(x, device="cuda"):
    return torch.as_tensor(np.asarray(x, np.int32)).to(device)


def random_cache(fmt, pages, g, hkv=4, ring=0, device="cuda"):
    """(k, v, k_dequant, v_dequant): pages (or rings) of N(0, 1)-like contents."""
    n = ring or 128
    if fmt == INT4:
        out = []
        for dims in (192, 128):
            codes = torch.randint(0, 16, (pages, hkv, n, dims), generator=g, device=device, dtype=torch.uint8)
            s = torch.rand((pages, hkv, n, dims // 32), generator=g, device=device) * 0.3 + 0.05
            out.append(int4_block(codes, s))
        return out[0], out[1], None, None
    k = torch.randn((pages, n, hkv, 192), generator=g, device=device)
    v = torch.randn((pages, n, hkv, 128), generator=g, device=device)
    if fmt == E4M3:
        kd = torch.rand(hkv, generator=g, device=device) * 0.1 + 0.02
        vd = torch.rand(hkv, generator=g, device=device) * 0.1 + 0.02
        return ((k / kd[:, None]).clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8),
                (v / vd[:, None]).clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8), kd, vd)
    kb = k.bfloat16()
    kb[..., :64] = k[..., :64].half().view(torch.bfloat16)
    return kb, v.bfloat16(), None, None
