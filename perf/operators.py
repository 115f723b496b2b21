"""Workloads of the operators that keep a long context's KV cache small: append to and decode over
a cache held in 4 bits, attention weights accumulated per cached slot, the selection of the slots
that stay, and the gather of those slots into other pages (or of a narrow cache into bf16).

`own` False: elementary torch operations.  `own` True: the library's calls.
"""
import math

import numpy as np
import torch

own = False

HQ, DK, DV, ROPE, PAGE = 64, 192, 128, 64, 128
SCALE = 1.0 / math.sqrt(192.0)
V_SCALE = 0.707
GLOBAL_BASE, SWA_BASE = 1e7, 1e4
BF16, E4M3, INT4 = 0, 1, 2
K_CODES, V_CODES = DK // 2, DV // 2  # bytes of 4-bit codes per slot
K_GROUPS, V_GROUPS = DK // 32, DV // 32  # fp16 scales per slot
K_SLOT, V_SLOT = K_CODES + 2 * K_GROUPS, V_CODES + 2 * V_GROUPS


# ------------------------------------------------------------------------------------- cases

def listed():
    return [
        # one short conversation: the latency of a single call
        dict(name="decode4_one", op="decode", B=1, q_len=1, lo=500, hi=500, ring=0),
        # a full serving batch over ragged long contexts (the repository's paged decode workload)
        dict(name="decode4_batch", op="decode", B=64, q_len=1, lo=4096, hi=65536, ring=0),
        # one very long context: the work of a few rows split over the whole GPU
        dict(name="decode4_long", op="decode", B=1, q_len=1, lo=131001, hi=131001, ring=0),
        # draft tokens of speculative decoding scored in one pass
        dict(name="decode4_drafts", op="decode", B=16, q_len=4, lo=1001, hi=16384, ring=0),
        # the sliding-window layers' rings (8 KV heads, sinks)
        dict(name="decode4_ring", op="decode", B=64, q_len=1, lo=200, hi=5000, ring=144),
        # one decode step of a batch as served: the new token's key and value stored, then attention
        dict(name="step4", op="step", B=48, q_len=1, lo=300, hi=8191, ring=0),
        # a prompt chunk stored in 4 bits and read back as bf16 pages for the next chunk's prefill
        dict(name="append4_chunk", op="append", B=3, lo=1500, hi=3000),
        # accumulated weights of a decode step, bf16 keys
        dict(name="weights_bf16", op="weights", fmt=BF16, B=32, q_len=1, lo=1000, hi=16384),
        # accumulated weights of the last drafts over long 4-bit contexts
        dict(name="weights_int4", op="weights", fmt=INT4, B=8, q_len=4, lo=4099, hi=65536),
        # eviction's selection in short and in long contexts
        dict(name="select_short", op="select", B=4, lo=700, hi=2500, keep=512, recent=64, first=4),
        dict(name="select_long", op="select", B=16, lo=40000, hi=131072, keep=16384, recent=1024, first=4),
        # the kept slots moved into fresh pages
        dict(name="gather_bf16", op="gather", fmt=BF16, B=16, lo=8000, hi=32768, keep=4000),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["decode", "decode", "decode", "step", "append", "weights", "select", "gather"])
    if op in ("decode", "step"):
        ring = rng.choice([0, 0, 128, 144, 512]) if op == "decode" else 0
        q_len = rng.choice([1, 1, 1, 2, 4, 7]) if op == "decode" else 1
        if ring and ring < 128 + q_len - 1:
            ring = 144
        hi = _log_int(rng, 300, 65536)
        B = max(1, min(_log_int(rng, 1, 64), 1 << 21 >> int(math.log2(hi * q_len))))
        return dict(op=op, B=B, q_len=q_len, lo=max(100, hi // rng.choice([1, 3, 10])), hi=hi, ring=ring)
    if op == "append":
        hi = _log_int(rng, 16, 4000)
        return dict(op=op, B=rng.randint(1, 4), lo=max(1, hi // rng.choice([1, 2, 5])), hi=hi)
    if op == "weights":
        hi = _log_int(rng, 300, 65536)
        return dict(op=op, fmt=rng.choice([BF16, E4M3, INT4]), B=max(1, min(_log_int(rng, 1, 32), (1 << 19) // hi)),
                    q_len=rng.choice([1, 1, 2, 5, 8]), lo=max(100, hi // rng.choice([1, 2, 8])), hi=hi)
    hi = _log_int(rng, 300, 131072 if op == "select" else 65536)
    B = max(1, min(_log_int(rng, 1, 64), (1 << 20) // hi))
    lo = max(20, hi // rng.choice([1, 2, 8]))
    keep = max(16, int(hi * rng.uniform(0.05, 0.9)))
    if op == "select":
        recent = rng.randint(0, keep // 2)
        return dict(op=op, B=B, lo=lo, hi=hi, keep=keep, recent=recent, first=rng.choice([0, 4, min(keep - recent, 7)]))
    keep = min(keep, 16000)
    return dict(op=op, fmt=rng.choice([BF16, E4M3, INT4]), B=max(1, min(B, (1 << 16) // keep)), lo=lo, hi=hi, keep=keep)


def _kv_heads(case):
    return 8 if case.get("ring") else 4


def work(case):
    """Bytes read and written once, and the flops."""
    op, B, lens = case["op"], case["B"], _lens(case)
    mean = float(lens.mean())
    hkv = _kv_heads(case)
    row = {BF16: 640, E4M3: 320, INT4: K_SLOT + V_SLOT}
    if op in ("decode", "step"):
        keys = hkv * float(np.minimum(lens, case["ring"] or case["hi"]).sum())
        q = B * case["q_len"] * HQ
        io = q * (DK * 2 + DV * 2 + 4)
        if op == "step":
            io += B * hkv * (DK + DV) * 2 + B * hkv * row[INT4]
        return dict(bytes=keys * row[INT4] + io, flops=2 * keys * (HQ // hkv) * case["q_len"] * (DK + DV))
    if op == "append":  # stored in 4 bits, read again and written as bf16
        return dict(bytes=B * mean * hkv * (640 + 2 * row[INT4] + 640), flops=0)
    if op == "weights":
        keys = B * hkv * mean
        kb = {BF16: 384, E4M3: 192, INT4: K_SLOT}[case["fmt"]]
        return dict(bytes=keys * (kb + 8) + B * case["q_len"] * HQ * (DK * 2 + 4),
                    flops=2 * keys * (HQ // hkv) * case["q_len"] * DK)
    kept = hkv * float(np.minimum(lens, case["keep"]).sum())
    if op == "select":
        return dict(bytes=B * hkv * mean * 4 + kept * 8, flops=0)
    return dict(bytes=kept * (2 * row[case["fmt"]] + 4), flops=0)


# ------------------------------------------------------------------------------------- inputs

def _lens(case, seed=None):
    """The case's context lengths; the seed says which sequence has which."""
    x = np.random.default_rng(17).integers(case["lo"], case["hi"] + 1, size=case["B"]).astype(np.int32)
    return x if seed is None else np.random.default_rng(seed).permutation(x)


def _pages(lens, r, spare=3):
    """A block table over a shuffled pool of pages, 0 behind each sequence's last page."""
    n = [-(-int(x) // PAGE) for x in lens]
    pool = r.permutation(sum(n) + spare).astype(np.int32)
    table = np.zeros((len(lens), max(n)), np.int32)
    at = 0
    for s, k in enumerate(n):
        table[s, :k] = pool[at:at + k]
        at += k
    return torch.from_numpy(table).cuda(), len(pool)


def _int4_cache(g, blocks, hkv, slots, slot_bytes, code_bytes):
    """Random codes 1..15 and fp16 scales as the groups of N(0, 1) rows give them (largest of 32
    over 7: about 0.3)."""
    nc, ns = slots * code_bytes, slots * (slot_bytes - code_bytes) // 2
    out = torch.empty((blocks, hkv, slots * slot_bytes), dtype=torch.uint8, device="cuda")
    c = torch.randint(0, 256, (blocks, hkv, nc), dtype=torch.uint8, device="cuda", generator=g)
    c |= ((c & 0x0F) == 0).to(torch.uint8)
    c |= ((c & 0xF0) == 0).to(torch.uint8) << 4
    out[..., :nc] = c
    s = torch.rand((blocks, hkv, ns), device="cuda", generator=g).mul_(0.2).add_(0.2).half()
    out[..., nc:] = s.view(torch.uint8)
    return out


def _cache(g, fmt, pages):
    """(k_cache, v_cache, k_dequant, v_dequant) of a paged cache of 4 KV heads."""
    if fmt == INT4:
        return (_int4_cache(g, pages, 4, PAGE, K_SLOT, K_CODES), _int4_cache(g, pages, 4, PAGE, V_SLOT, V_CODES), None, None)
    if fmt == E4M3:
        k = torch.randn((pages, PAGE, 4, DK), device="cuda", generator=g).mul_(20).to(torch.float8_e4m3fn).view(torch.uint8)
        v = torch.randn((pages, PAGE, 4, DV), device="cuda", generator=g).mul_(20).to(torch.float8_e4m3fn).view(torch.uint8)
        return k, v, torch.full((4,), 0.05, device="cuda"), torch.full((4,), 0.04, device="cuda")
    k = torch.randn((pages, PAGE, 4, DK), device="cuda", generator=g, dtype=torch.bfloat16)
    k[..., :ROPE] = torch.randn((pages, PAGE, 4, ROPE), device="cuda", generator=g).half().view(torch.bfloat16)
    return k, torch.randn((pages, PAGE, 4, DV), device="cuda", generator=g, dtype=torch.bfloat16), None, None


def _bf16(g, *shape):
    return torch.randn(shape, device="cuda", generator=g, dtype=torch.bfloat16)


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    r = np.random.default_rng(seed)
    op, B = case["op"], case["B"]
    lens = _lens(case, seed)
    st = dict(case=case, lens=torch.from_numpy(lens).cuda(), max_len=int(lens.max()), B=B)
    if op in ("decode", "step"):
        ql, hkv = case["q_len"], _kv_heads(case)
        st["q"] = _bf16(g, B * ql, HQ, DK)
        if case["ring"]:
            st["k"] = _int4_cache(g, B, hkv, case["ring"], K_SLOT, K_CODES)
            st["v"] = _int4_cache(g, B, hkv, case["ring"], V_SLOT, V_CODES)
            st["sink"] = torch.randn(HQ, device="cuda", generator=g)
            st["table"], st["pages"] = None, 0
        else:
            st["table"], st["pages"] = _pages(lens, r)
            st["k"], st["v"], _, _ = _cache(g, INT4, st["pages"])
            st["sink"] = None
        if op == "step":
            st["k_new"], st["v_new"] = _bf16(g, B, hkv, DK), _bf16(g, B, hkv, DV)
            st["pos"], st["seq"] = st["lens"] - 1, torch.arange(B, dtype=torch.int32, device="cuda")
        st["workspace"] = torch.empty(64 << 20, dtype=torch.uint8, device="cuda")  # a serving loop's scratch
        return st
    if op == "append":
        n = int(lens.sum())
        st["table"], st["pages"] = _pages(lens, r, spare=0)
        st["k_new"], st["v_new"] = _bf16(g, n, 4, DK), _bf16(g, n, 4, DV)
        st["pos"] = torch.from_numpy(np.concatenate([np.arange(x) for x in lens]).astype(np.int32)).cuda()
        st["seq"] = torch.from_numpy(np.repeat(np.arange(B), lens).astype(np.int32)).cuda()
        st["k"] = torch.zeros((st["pages"], 4, PAGE * K_SLOT), dtype=torch.uint8, device="cuda")
        st["v"] = torch.zeros((st["pages"], 4, PAGE * V_SLOT), dtype=torch.uint8, device="cuda")
        st["table_out"], st["pages_out"] = _pages(lens, r, spare=0)
        st["k_out"] = torch.zeros((st["pages_out"], PAGE, 4, DK), dtype=torch.bfloat16, device="cuda")
        st["v_out"] = torch.zeros((st["pages_out"], PAGE, 4, DV), dtype=torch.bfloat16, device="cuda")
        return st
    if op == "weights":
        ql = case["q_len"]
        st["table"], st["pages"] = _pages(lens, r)
        st["k"], _, st["k_dequant"], _ = _cache(g, case["fmt"], st["pages"])
        st["q"] = _bf16(g, B * ql, HQ, DK)
        z = _logits(st["q"], _paged_keys(st, case["fmt"]), st["lens"], ql, GLOBAL_BASE)
        z = z.masked_fill_(~_visible(st["lens"], ql, z.shape[-1])[:, None, :, None, :], -math.inf)
        # the decode call's log-sum-exp of the same queries
        st["lse"] = torch.logsumexp(z, -1).permute(0, 2, 1, 3).reshape(B * ql, HQ).contiguous()
        # what earlier steps left behind
        st["scores"] = torch.rand((B, 4, z.shape[-1]), device="cuda", generator=g).mul_(0.01)
        return st
    if op == "select":
        # accumulated weights: most slots small, a few large, and ties among what was never attended
        x = torch.rand((B, 4, st["max_len"]), device="cuda", generator=g)
        st["scores"] = torch.where(x < 0.2, torch.zeros_like(x), torch.exp(-8 * x))
        return st
    st["table"], st["pages"] = _pages(lens, r)
    st["k"], st["v"], st["k_dequant"], st["v_dequant"] = _cache(g, case["fmt"], st["pages"])
    kept = np.minimum(lens, case["keep"])
    cap = int(kept.max())
    # the kept slots, ascending, another choice for every head
    x = torch.rand((B, 4, st["max_len"]), device="cuda", generator=g)
    t = torch.arange(st["max_len"], device="cuda")
    x = torch.where(t < st["lens"][:, None, None], x, torch.full_like(x, 2.0))
    idx = x.argsort(-1)[..., :cap]
    st["counts"] = torch.from_numpy(kept.astype(np.int32)).cuda()
    j = torch.arange(cap, device="cuda")
    idx = torch.where(j < st["counts"][:, None, None], idx, torch.full_like(idx, 1 << 30)).sort(-1).values
    st["idx"] = torch.where(idx < 1 << 30, idx, torch.full_like(idx, -1)).int().contiguous()
    st["table_out"], st["pages_out"] = _pages(kept, r, spare=0)
    if case["fmt"] == INT4:
        st["k_out"] = torch.zeros((st["pages_out"], 4, PAGE * K_SLOT), dtype=torch.uint8, device="cuda")
        st["v_out"] = torch.zeros((st["pages_out"], 4, PAGE * V_SLOT), dtype=torch.uint8, device="cuda")
    else:
        st["k_out"] = torch.zeros((st["pages_out"], PAGE, 4, DK), dtype=st["k"].dtype, device="cuda")
        st["v_out"] = torch.zeros((st["pages_out"], PAGE, 4, DV), dtype=st["v"].dtype, device="cuda")
    return st


# ------------------------------------------------------------------------------------- plain form

def _cos_sin(pos, base):
    """float32 cos and sin of the rotary angles, the angles in 64 bits: [..., 32]."""
    inv = base ** (-2.0 * torch.arange(ROPE // 2, dtype=torch.float64, device=pos.device) / ROPE)
    a = pos.double()[..., None] * inv
    return a.cos().float(), a.sin().float()


def _rotate(x, pos, base):
    """float32 rows [n, heads, 192] with dims 0..63 rotated at pos [n]."""
    x = x.float()
    c, s = _cos_sin(pos, base)
    c, s = c[:, None], s[:, None]
    a, b = x[..., :32], x[..., 32:64]
    return torch.cat([a * c - b * s, b * c + a * s, x[..., 64:]], -1)


def _nibbles(codes):
    """[..., n] bytes -> [..., 2 n] float32 in -8..7, the low nibble first."""
    return torch.stack([codes & 15, codes >> 4], -1).flatten(-2).float().sub_(8)


def _unpack(block, slots, code_bytes, key):
    """[..., slots * slot_bytes] blocks -> [..., slots, dims] float32."""
    n = slots * code_bytes
    codes = block[..., :n].unflatten(-1, (slots, code_bytes))
    if key:  # words of 8 dims: word w sits at (w % 4) * 6 + w // 4
        codes = codes.unflatten(-1, (4, 6, 4)).transpose(-3, -2).flatten(-3)
    scales = block[..., n:].contiguous().view(torch.half).unflatten(-1, (slots, code_bytes // 16))
    x = _nibbles(codes).unflatten(-1, (-1, 32))
    return x.mul_(scales.float()[..., None]).flatten(-2)


def _quantise(x):
    """Rows [..., d] float32 -> (codes in -7..7, float32 scale per group of 32)."""
    g = x.unflatten(-1, (-1, 32))
    s = (g.abs().amax(-1) / 7.0).half().float()
    n = torch.where(s[..., None] > 0, torch.round(g / s[..., None]).clamp(-7, 7), torch.zeros_like(g))
    return n, s


def _fake_quant(x):
    n, s = _quantise(x)
    return (n * s[..., None]).flatten(-2)


def _paged_int4(cache, table, code_bytes, key):
    """[B, Hkv, slots, dims] float32 of every page in the block table."""
    rows = cache[table.long()].transpose(1, 2)
    x = _unpack(rows, PAGE, code_bytes, key)
    return x.flatten(2, 3)


def _wide_keys(k):
    """bf16 cache rows (dims 0..63 hold fp16) -> float32."""
    return torch.cat([k[..., :ROPE].contiguous().view(torch.half).float(), k[..., ROPE:].float()], -1)


def _paged_keys(st, fmt):
    if fmt == INT4:
        return _paged_int4(st["k"], st["table"], K_CODES, True)
    rows = st["k"][st["table"].long()].flatten(1, 2).transpose(1, 2)
    if fmt == BF16:
        return _wide_keys(rows)
    return rows.contiguous().view(torch.float8_e4m3fn).float() * st["k_dequant"][None, :, None, None]


def _logits(q, k, lens, q_len, base):
    """[B, Hkv, q_len, G, slots] scaled logits of the last q_len tokens of each sequence."""
    B, hkv = k.shape[:2]
    pos = (lens[:, None] - q_len + torch.arange(q_len, device=lens.device)).flatten()
    qr = _rotate(q, pos, base).view(B, q_len, hkv, HQ // hkv, DK).transpose(1, 2).reshape(B, hkv, -1, DK)
    return (qr @ k.transpose(-1, -2)).mul_(SCALE).view(B, hkv, q_len, HQ // hkv, -1)


def _visible(lens, q_len, slots):
    """[B, q_len, slots]: draft i sees the slots up to its own."""
    last = lens[:, None] - q_len + torch.arange(q_len, device=lens.device)
    return torch.arange(slots, device=lens.device) <= last[..., None]


def _attend(z, vis, v, sink):
    """Softmax over the visible slots, a sink logit in the denominator, times V."""
    B, hkv, ql, G, _ = z.shape
    z = z.masked_fill_(~vis[:, None, :, None, :], -math.inf)
    m = z.amax(-1, keepdim=True)
    if sink is not None:
        sk = sink.view(1, hkv, 1, G, 1)
        m = torch.maximum(m, sk)
    e = z.sub_(m).exp_()
    l = e.sum(-1, keepdim=True)
    if sink is not None:
        l = l + (sk - m).exp()
    o = (e.view(B, hkv, ql * G, -1) @ v).view(B, hkv, ql, G, DV) / l * V_SCALE
    lse = (m + l.log())[..., 0]
    return o.transpose(1, 2).reshape(B * ql, HQ, DV).bfloat16(), lse.transpose(1, 2).reshape(B * ql, HQ)


def _plain_decode(st):
    case, lens, ql = st["case"], st["lens"], st["case"]["q_len"]
    if case["ring"]:
        R = case["ring"]
        k, v = _unpack(st["k"], R, K_CODES, True), _unpack(st["v"], R, V_CODES, False)
        z = _logits(st["q"], k, lens, ql, SWA_BASE)
        slot = torch.arange(R, device=lens.device)
        at = lens[:, None] - R + (slot - lens[:, None]) % R  # position that each slot holds
        mine = lens[:, None] - ql + torch.arange(ql, device=lens.device)
        back = mine[..., None] - at[:, None, :]
        vis = (back >= 0) & (back < R - ql + 1) & (at >= 0)[:, None, :]
        return _attend(z, vis, v, st["sink"])
    k, v = _paged_int4(st["k"], st["table"], K_CODES, True), _paged_int4(st["v"], st["table"], V_CODES, False)
    if case["op"] == "step":
        b, p = st["seq"].long(), st["pos"].long()
        k[b, :, p] = _fake_quant(_rotate(st["k_new"], st["pos"], GLOBAL_BASE))
        v[b, :, p] = _fake_quant(st["v_new"].float())
    z = _logits(st["q"], k, lens, ql, GLOBAL_BASE)
    del k
    return _attend(z, _visible(lens, ql, z.shape[-1]), v, None)


def _plain_append(st):
    k = _fake_quant(_rotate(st["k_new"], st["pos"], GLOBAL_BASE))
    v = _fake_quant(st["v_new"].float())
    page = st["table_out"][st["seq"].long(), (st["pos"] // PAGE).long()].long()
    slot = (st["pos"] % PAGE).long()
    n = st["pages_out"]
    rot = torch.zeros((n, PAGE, 4, ROPE), dtype=torch.half, device="cuda")
    rest = torch.zeros((n, PAGE, 4, DK - ROPE), dtype=torch.bfloat16, device="cuda")
    val = torch.zeros((n, PAGE, 4, DV), dtype=torch.bfloat16, device="cuda")
    rot[page, slot] = k[..., :ROPE].half()
    rest[page, slot] = k[..., ROPE:].bfloat16()
    val[page, slot] = v.bfloat16()
    return rot, rest, val


def _plain_weights(st):
    ql = st["case"]["q_len"]
    B = st["B"]
    z = _logits(st["q"], _paged_keys(st, st["case"]["fmt"]), st["lens"], ql, GLOBAL_BASE)
    lse = st["lse"].view(B, ql, 4, HQ // 4).transpose(1, 2)
    p = (z - lse[..., None]).exp_()
    p = p.masked_fill_(~_visible(st["lens"], ql, z.shape[-1])[:, None, :, None, :], 0.0)
    return st["scores"].add_(p.sum((2, 3)))


def _plain_select(st):
    case, s, lens = st["case"], st["scores"], st["lens"][:, None, None]
    keep, recent, first = case["keep"], case["recent"], case["first"]
    t = torch.arange(s.shape[-1], device=s.device).expand(s.shape)
    order = torch.sort(torch.nan_to_num(s, nan=-math.inf, posinf=math.inf, neginf=-math.inf), dim=-1, descending=True,
                       stable=True).indices
    rank = torch.where(t >= lens, 2, torch.where((t < first) | (t >= lens - recent), 0, 1))
    rank = rank.gather(-1, order)
    order = order.gather(-1, torch.sort(rank, dim=-1, stable=True).indices)[..., :keep]
    counts = st["lens"].clamp(max=keep)
    far = s.shape[-1]
    pad = torch.arange(order.shape[-1], device=s.device) >= counts[:, None, None]
    order = torch.where(pad, torch.full_like(order, far), order).sort(-1).values
    vals = s.gather(-1, order.clamp(max=far - 1)).masked_fill(pad, 0.0)
    idx = torch.where(pad, torch.full_like(order, -1), order).int()
    if idx.shape[-1] < keep:
        more = keep - idx.shape[-1]
        idx = torch.nn.functional.pad(idx, (0, more), value=-1)
        vals = torch.nn.functional.pad(vals, (0, more))
    return idx, counts, vals


def _values(st, k, v, fmt):
    """A cache's contents as the values it stands for."""
    if fmt == INT4:
        return _unpack(k, PAGE, K_CODES, True).half(), _unpack(v, PAGE, V_CODES, False).half()
    if fmt == E4M3:
        return k.view(torch.float8_e4m3fn), v.view(torch.float8_e4m3fn)
    return k[..., :ROPE].view(torch.half), k[..., ROPE:], v


def _plain_gather(st):
    fmt = st["case"]["fmt"]
    B, H, cap = st["idx"].shape
    j = torch.arange(cap, device="cuda").expand(B, H, cap)
    b = torch.arange(B, device="cuda")[:, None, None].expand(B, H, cap)
    h = torch.arange(H, device="cuda")[None, :, None].expand(B, H, cap)
    ok = st["idx"] >= 0
    j, b, h, i = j[ok], b[ok], h[ok], st["idx"][ok].long()
    src, dst = st["table"][b, i // PAGE].long(), st["table_out"][b, j // PAGE].long()
    n = st["pages_out"]

    def move(cache, width, slot_bytes):
        if fmt != INT4:
            out = torch.zeros((n, PAGE, H, width), dtype=cache.dtype, device="cuda")
            out[dst, j % PAGE, h] = cache[src, i % PAGE, h]
            return out
        out = torch.zeros((n, H, PAGE * slot_bytes), dtype=torch.uint8, device="cuda")
        codes = width // 2
        a, z = out[..., :PAGE * codes].view(n, H, PAGE, codes), out[..., PAGE * codes:].view(n, H, PAGE, -1)
        ca = cache[..., :PAGE * codes].view(cache.shape[0], H, PAGE, codes)
        cz = cache[..., PAGE * codes:].view(cache.shape[0], H, PAGE, -1)
        a[dst, h, j % PAGE] = ca[src, h, i % PAGE]
        z[dst, h, j % PAGE] = cz[src, h, i % PAGE]
        return out

    return move(st["k"], DK, K_SLOT), move(st["v"], DV, V_SLOT)


# ------------------------------------------------------------------------------------- the library

def _own_append(st):
    import global_attention_attn_b200 as M
    M.mimo_kv_append(st["k_new"], st["v_new"], st["pos"], st["seq"], rope_base=GLOBAL_BASE, cache_kind=M.MIMO_CACHE_PAGED,
                     k_cache=st["k"], v_cache=st["v"], num_seqs=st["B"], block_table=st["table"], num_pages=st["pages"],
                     cache_dtype=M.MIMO_DTYPE_INT4)


def _own_decode(st):
    import global_attention_attn_b200 as M
    case = st["case"]
    ring = case["ring"]
    return M.mimo_attn_decode(
        st["q"], st["lens"], max_seq_len=st["max_len"], num_kv_heads=_kv_heads(case),
        rope_base=SWA_BASE if ring else GLOBAL_BASE, window=ring - case["q_len"] + 1 if ring else 0,
        cache_kind=M.MIMO_CACHE_RING if ring else M.MIMO_CACHE_PAGED, k_cache=st["k"], v_cache=st["v"],
        block_table=st["table"], num_pages=st["pages"], sink=st["sink"], workspace=st["workspace"],
        cache_dtype=M.MIMO_DTYPE_INT4, ring_slots=ring, q_len=case["q_len"])


def _own_weights(st):
    import global_attention_attn_b200 as M
    case = st["case"]
    return M.mimo_attn_weights(st["q"], st["lse"], st["scores"], st["lens"], max_seq_len=st["max_len"], num_kv_heads=4,
                               rope_base=GLOBAL_BASE, k_cache=st["k"], block_table=st["table"], num_pages=st["pages"],
                               cache_dtype=case["fmt"], k_dequant=st["k_dequant"], q_len=case["q_len"])


def _own_gather(st, fmt, out_fmt):
    import global_attention_attn_b200 as M
    M.mimo_kv_gather(st["k"], st["v"], st["table"], st["k_out"], st["v_out"], st["table_out"],
                     st.get("counts", st["lens"]), idx=st.get("idx"), num_kv_heads=4, num_pages=st["pages"],
                     num_pages_out=st["pages_out"], cache_dtype=fmt, out_dtype=out_fmt, k_dequant=st.get("k_dequant"),
                     v_dequant=st.get("v_dequant"))


def run(st):
    op = st["case"]["op"]
    if op in ("decode", "step"):
        if not own:
            return _plain_decode(st)
        if op == "step":
            _own_append(st)
        return _own_decode(st)
    if op == "append":
        if not own:
            return _plain_append(st)
        _own_append(st)
        _own_gather(st, INT4, BF16)
        return _values(st, st["k_out"], st["v_out"], BF16)
    if op == "weights":
        return _own_weights(st) if own else _plain_weights(st)
    if op == "select":
        if not own:
            return _plain_select(st)
        import global_attention_attn_b200 as M
        return M.mimo_kv_select(st["scores"], st["lens"], max_seq_len=st["max_len"], keep=st["case"]["keep"],
                                recent=st["case"]["recent"], first=st["case"]["first"])
    fmt = st["case"]["fmt"]
    if not own:
        return _values(st, *_plain_gather(st), fmt)
    _own_gather(st, fmt, fmt)
    return _values(st, st["k_out"], st["v_out"], fmt)


# ------------------------------------------------------------------------------------- 64 bits

def _x_rows(cache, page, heads, dims, fmt, key, dequant, slots=PAGE):
    """float64 [heads, slots, dims] of one page (or ring) from the format's definition: each
    element's byte, nibble and group scale looked up by its dim."""
    if fmt == BF16:
        x = cache[page].transpose(0, 1)
        if key:
            return torch.cat([x[..., :64].contiguous().view(torch.half).double(), x[..., 64:].double()], -1)
        return x.double()
    if fmt == E4M3:
        return cache[page].transpose(0, 1).contiguous().view(torch.float8_e4m3fn).double() * dequant.double().view(-1, 1, 1)
    d = torch.arange(dims, device="cuda")
    w = d // 8
    word = (w % 4) * 6 + w // 4 if key else w
    byte = (word * 4 + d % 8 // 2)[None, :] + torch.arange(slots, device="cuda")[:, None] * (dims // 2)
    blk = cache[page]
    code = (blk[:, byte.flatten()].view(heads, slots, dims).int() >> (4 * (d % 2)).int()) & 15
    scale = blk[:, slots * dims // 2:].contiguous().view(torch.half).view(heads, slots, dims // 32).double()
    return (code.double() - 8) * scale[:, :, d // 32]


def _x_rotated(x, pos, base):
    x = x.double()
    out = x.clone()
    for j in range(32):
        a = pos.double() * base ** (-j / 32.0)
        c, s = a.cos()[:, None], a.sin()[:, None]
        out[:, :, j] = x[:, :, j] * c - x[:, :, j + 32] * s
        out[:, :, j + 32] = x[:, :, j + 32] * c + x[:, :, j] * s
    return out


def _x_quant(x):
    g = x.reshape(*x.shape[:-1], -1, 32)
    s = (g.abs().max(-1, keepdim=True).values / 7).half().double()
    return torch.where(s > 0, torch.round(g / s).clamp(-7, 7) * s, torch.zeros_like(g)).reshape(x.shape)


def exact(case, seed):
    st = prepare(case, seed)
    op, B, ql = case["op"], case["B"], case.get("q_len", 1)
    lens = st["lens"].tolist()
    if op in ("decode", "step", "weights"):
        ring, hkv = case.get("ring", 0), _kv_heads(case)
        fmt = case.get("fmt", INT4)
        base = SWA_BASE if ring else GLOBAL_BASE
        G = HQ // hkv
        outs, lses = [], []
        scores = st["scores"].double() if op == "weights" else None
        for b in range(B):
            n = lens[b]
            if ring:
                lo = max(0, n - ring)
                at = torch.arange(lo, n, device="cuda")
                k = _x_rows(st["k"], b, hkv, DK, INT4, True, None, ring)[:, at % ring]
                v = _x_rows(st["v"], b, hkv, DV, INT4, False, None, ring)[:, at % ring]
            else:
                at = torch.arange(n, device="cuda")
                pages = st["table"][b].tolist()[:-(-n // PAGE)]
                k = torch.cat([_x_rows(st["k"], p, hkv, DK, fmt, True, st.get("k_dequant")) for p in pages], 1)[:, :n]
                if op != "weights":
                    v = torch.cat([_x_rows(st["v"], p, hkv, DV, fmt, False, None) for p in pages], 1)[:, :n]
            if op == "step":
                k[:, n - 1] = _x_quant(_x_rotated(st["k_new"][b:b + 1], st["pos"][b:b + 1], base))[0]
                v[:, n - 1] = _x_quant(st["v_new"][b].double())
            for i in range(ql):
                me = n - ql + i
                q = _x_rotated(st["q"][b * ql + i][None], torch.tensor([me], device="cuda"), base)[0].view(hkv, G, DK)
                see = (at <= me) & (at > me - (ring - ql + 1) if ring else at >= 0)
                z = torch.einsum("hgd,htd->hgt", q, k) / math.sqrt(192.0)
                z[:, :, ~see] = -math.inf
                if op == "weights":
                    scores[b, :, :n] += torch.exp(z - st["lse"][b * ql + i].double().view(hkv, G, 1)).sum(1)
                    continue
                a = torch.logsumexp(z, -1)
                if st["sink"] is not None:
                    a = torch.logaddexp(a, st["sink"].double().view(hkv, G))
                outs.append((torch.exp(z - a[..., None]) @ v).reshape(HQ, DV) * V_SCALE)
                lses.append(a.reshape(HQ))
        return scores if op == "weights" else (torch.stack(outs), torch.stack(lses))
    if op == "append":
        k = _x_quant(_x_rotated(st["k_new"], st["pos"], GLOBAL_BASE))
        v = _x_quant(st["v_new"].double())
        rot = torch.zeros((st["pages_out"], PAGE, 4, ROPE), dtype=torch.float64, device="cuda")
        rest, val = torch.zeros_like(rot).repeat(1, 1, 1, 2), torch.zeros_like(rot).repeat(1, 1, 1, 2)
        at = 0
        for b in range(B):
            for t in range(0, lens[b], PAGE):
                m, p = min(PAGE, lens[b] - t), int(st["table_out"][b, t // PAGE])
                rot[p, :m], rest[p, :m], val[p, :m] = k[at:at + m, :, :ROPE], k[at:at + m, :, ROPE:], v[at:at + m]
                at += m
        return rot, rest, val
    if op == "select":  # the scores kept, by a sort of (class, score, slot) on the host
        x = torch.nan_to_num(st["scores"], nan=-math.inf).double().cpu().numpy()
        vals = np.zeros((B, 4, case["keep"]))
        for b in range(B):
            t = np.arange(lens[b])
            forced = (t < case["first"]) | (t >= lens[b] - case["recent"])
            for h in range(4):
                row = x[b, h, :lens[b]]
                kept = np.sort(np.lexsort((t, -row, ~forced))[:case["keep"]])
                vals[b, h, :len(kept)] = row[kept]
        return None, None, torch.from_numpy(vals)
    return None  # a gather moves bytes
