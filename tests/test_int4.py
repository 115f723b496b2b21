"""The 4-bit cache: quantising append, decode and draft verification over pages and rings,
against float64 on the values the cache stands for; refusals and layout on the CPU."""
import ctypes as C

import numpy as np
import pytest
import torch

import global_attention_attn_b200 as M
from tests import cache_ref as R

gpu = pytest.mark.gpu
PAGED, RING = M.MIMO_CACHE_PAGED, M.MIMO_CACHE_RING


def gen(seed, device="cuda"):
    return torch.Generator(device=device).manual_seed(seed)


# ----------------------------------------------------------------------------- CPU

def test_layout_round_trip():
    g = torch.Generator().manual_seed(1)
    for dims, slot in ((192, M.MIMO_INT4_K_SLOT_BYTES), (128, M.MIMO_INT4_V_SLOT_BYTES)):
        codes = torch.randint(0, 16, (2, 3, 16, dims), generator=g, dtype=torch.uint8)
        s = torch.rand((2, 3, 16, dims // 32), generator=g).half()
        b = R.int4_block(codes, s)
        assert b.shape == (2, 3, 16 * slot)
        want = (codes.double() - 8) * s.double().repeat_interleave(32, -1)
        assert torch.equal(R.int4_values(b, 16, dims), want)


def test_quantise_is_within_half_a_step():
    x = torch.randn(500, 192, generator=torch.Generator().manual_seed(2))
    c, s = R.int4_quantise(x)
    assert int(c.min()) >= 1 and int(c.max()) <= 15
    sd = s.double().repeat_interleave(32, -1)
    # half a step, and (the fp16 scale may round down by 2^-11) a clamped 7 of 7 (1 + 2^-11)
    assert (((c.double() - 8) * sd - x.double()).abs() <= sd * (0.5 + 7 * 2.0 ** -11)).all()


def _decode_args(**kw):
    a = M.MimoDecodeArgs()
    a.layer = M.make_layer(kw.pop("hkv", 4), 1e7, kw.pop("window", 0))
    p = 1 << 20  # an address that is never read: every check here is on the host
    a.batch, a.max_seq_len, a.cache_kind, a.cache_dtype = 2, 300, PAGED, M.MIMO_DTYPE_INT4
    a.q = a.seq_lens = a.k_cache = a.v_cache = a.out = a.block_table = a.workspace = p
    a.workspace_bytes, a.max_pages, a.num_pages, a.q_len = 64 << 20, 3, 8, 1
    for k, v in kw.items():
        setattr(a, k, v)
    return a


@pytest.mark.parametrize("kw, code, word", [
    (dict(k_dequant=1 << 20), M.MIMO_ERR_INVALID_ARG, "must be NULL"),
    (dict(v_dequant=1 << 20), M.MIMO_ERR_INVALID_ARG, "must be NULL"),
    (dict(cache_dtype=3), M.MIMO_ERR_INVALID_ARG, "cache_dtype"),
    (dict(q_len=9), M.MIMO_ERR_INVALID_ARG, "q_len"),
    (dict(workspace=None), M.MIMO_ERR_WORKSPACE, "workspace"),
    (dict(workspace_bytes=100), M.MIMO_ERR_WORKSPACE, "workspace"),
    (dict(workspace=(1 << 20) + 8), M.MIMO_ERR_INVALID_ARG, "aligned"),
    (dict(max_pages=2), M.MIMO_ERR_INVALID_ARG, "max_pages"),
    (dict(positions=(1 << 20) + 4), M.MIMO_ERR_INVALID_ARG, "positions"),
    (dict(positions=1 << 20, window=100), M.MIMO_ERR_INVALID_ARG, "positions"),
    (dict(positions=1 << 20, window=100, cache_kind=RING, hkv=8), M.MIMO_ERR_INVALID_ARG, "positions"),
    (dict(cache_kind=RING, hkv=8), M.MIMO_ERR_INVALID_ARG, "ring"),
    (dict(v_cache=None), M.MIMO_ERR_INVALID_ARG, "v_cache"),
])
def test_decode_refusals(kw, code, word):
    a = _decode_args(**kw)
    assert M.lib().mimo_attn_decode(C.byref(a), None) == code
    assert word in M.lib().mimo_last_error().decode()


@pytest.mark.parametrize("kw, word", [
    (dict(k_dequant=1 << 20), "must be NULL"),
    (dict(slots=1 << 20, cache_kind=RING), "slots"),
    (dict(slots=(1 << 20) + 4), "slots"),
    (dict(cache_dtype=7), "cache_dtype"),
])
def test_append_refusals(kw, word):
    a = M.MimoAppendArgs()
    p = 1 << 20
    a.num_tokens, a.num_kv_heads, a.head_dim_qk, a.head_dim_v, a.rope_dim, a.rope_base = 2, 4, 192, 128, 64, 1e7
    a.k_new = a.v_new = a.pos = a.seq_idx = a.k_cache = a.v_cache = a.block_table = p
    a.cache_kind, a.num_seqs, a.max_pages, a.num_pages, a.cache_dtype = PAGED, 2, 3, 8, M.MIMO_DTYPE_INT4
    for k, v in kw.items():
        setattr(a, k, v)
    assert M.lib().mimo_kv_append(C.byref(a), None) == M.MIMO_ERR_INVALID_ARG
    assert word in M.lib().mimo_last_error().decode()


def test_workspace_size():
    size = M.lib().mimo_attn_decode_int4_workspace_size
    assert size(4, 1, 5000, 8, 128, RING) == 0
    assert size(4, 1, 200, 4, 0, PAGED) == 0  # units of up to 8 tiles stay whole
    assert size(4, 1, 5000, 5, 0, PAGED) == 0 and size(4, 9, 5000, 4, 0, PAGED) == 0
    for q_len in range(1, 9):
        for hkv in (4, 8):
            for batch in (1, 64, 5000):
                for n in (300, 70000, 1 << 20):
                    assert 0 < size(batch, q_len, n, hkv, 0, PAGED) <= 20 << 20


# ----------------------------------------------------------------------------- append

def _append(k_new, v_new, pos, seq, k, v, base, **kw):
    M.mimo_kv_append(k_new, v_new, pos, seq, rope_base=base, k_cache=k, v_cache=v, cache_dtype=M.MIMO_DTYPE_INT4, **kw)


def _check_rows(got, want32, dims):
    """Stored values against the rule applied to the float64 rows: the same scale to one fp16
    step and the same code, but where the fp32 rotation moved a quotient over a border."""
    c, s = R.int4_quantise(want32.float())
    sd = s.double().repeat_interleave(32, -1)
    exact = (c.double() - 8) * sd
    step = sd * (1 + 2.0 ** -9)
    err = (got - exact).abs()
    assert (err <= step + 7 * sd * 2.0 ** -10).all()
    assert float((err > sd * 2.0 ** -6).double().mean()) < 1e-3
    # and always a valid rounding of the input
    assert ((got - want32).abs() <= sd * (0.5 + 7 * 2.0 ** -10) + 1e-5 * want32.abs().max()).all()


@gpu
@pytest.mark.parametrize("hkv, ring", [(4, 0), (8, 0), (8, 144), (8, 512)])
def test_append(hkv, ring):
    g, r = gen(3), np.random.default_rng(3)
    # (two tokens of one call must not share a slot: a ring takes at most its slots)
    lens = [1, 100, 128] if ring else [1, 130, 257]
    n = sum(lens)
    kn = torch.randn((n, hkv, 192), generator=g, device="cuda").mul_(3).bfloat16()
    vn = torch.randn((n, hkv, 128), generator=g, device="cuda").bfloat16()
    kn[5], vn[7] = 0, 0           # groups without a scale
    kn[9, 0, 64:96] = 1e-6        # a scale that is a subnormal of fp16
    seq = R.i32(np.repeat(np.arange(3), lens))
    pos = R.i32(np.concatenate([np.arange(x) + (1000 if i == 1 and ring else 0) for i, x in enumerate(lens)]))
    base = 1e4 if ring else 1e7
    if ring:
        k, v = M.empty_int4_cache(3, hkv, ring)
        _append(kn, vn, pos, seq, k, v, base, cache_kind=RING, num_seqs=3, ring_slots=ring)
    else:
        table, pages = R.table_of(lens, r)
        k, v = M.empty_int4_cache(pages, hkv)
        _append(kn, vn, pos, seq, k, v, base, cache_kind=PAGED, num_seqs=3, block_table=table, num_pages=pages)
    assert M.status_poll() == 0
    want_k, want_v = R.rotate(kn, pos, base), vn.double()
    kv, vv = R.slots_of(k, R.INT4, 192), R.slots_of(v, R.INT4, 128)
    at = 0
    for s, m in enumerate(lens):
        if ring:
            rows = torch.arange(at, at + m, device="cuda")
            slot = pos[rows].long() % ring
            gk, gv = kv[s][:, slot], vv[s][:, slot]
        else:
            rows = torch.arange(at, at + m, device="cuda")
            gk, gv = R.pages_of(kv, table[s], m), R.pages_of(vv, table[s], m)
        _check_rows(gk.transpose(0, 1), want_k[rows], 192)
        _check_rows(gv.transpose(0, 1), want_v[rows], 128)
        at += m


@gpu
def test_append_slots_and_skips():
    """`slots` places a token elsewhere than its rotary position says; tokens outside the cache
    are skipped and reported, and no other byte changes."""
    g = gen(4)
    kn, vn = (torch.randn((4, 4, d), generator=g, device="cuda").bfloat16() for d in (192, 128))
    table = R.i32([[2, 0], [1, -1]])
    k, v = M.empty_int4_cache(3, 4)
    k0, v0 = k.clone(), v.clone()
    kw = dict(cache_kind=PAGED, num_seqs=2, block_table=table, num_pages=3)
    # token 0 -> sequence 0 slot 130; 1 -> sequence 1 slot 128 (page -1); 2 -> slot < 0; 3 -> sequence 5
    _append(kn, vn, R.i32([9000, 1, 2, 3]), R.i32([0, 1, 0, 5]), k, v, 1e7, slots=R.i32([130, 128, -1, 0]), **kw)
    assert M.status_poll() == M.MIMO_STATUS_BAD_INDEX
    _check_rows(R.slots_of(k, R.INT4, 192)[0][:, 2][None], R.rotate(kn[:1], R.i32([9000]), 1e7), 192)
    own = torch.zeros_like(k, dtype=torch.bool)
    own[0, :, 2 * 96:3 * 96] = True
    own[0, :, 128 * 96 + 2 * 12:128 * 96 + 3 * 12] = True
    assert torch.equal(k[~own], k0[~own])
    own = torch.zeros_like(v, dtype=torch.bool)
    own[0, :, 2 * 64:3 * 64] = True
    own[0, :, 128 * 64 + 2 * 8:128 * 64 + 3 * 8] = True
    assert torch.equal(v[~own], v0[~own])


@gpu
def test_append_range_is_reported():
    kn, vn = torch.ones((3, 4, 192), device="cuda").bfloat16(), torch.ones((3, 4, 128), device="cuda").bfloat16()
    kn[0, 1, 70], vn[1, 0, 3], vn[2, 2, 127] = 1e6, 1e4, float("inf")
    k, v = M.empty_int4_cache(1, 4)
    _append(kn, vn, R.i32([0, 1, 2]), R.i32([0, 0, 0]), k, v, 1e7, cache_kind=PAGED, num_seqs=1,
            block_table=R.i32([[0]]), num_pages=1)
    assert M.status_poll() == M.MIMO_STATUS_RANGE
    kv, vv = R.slots_of(k, R.INT4, 192), R.slots_of(v, R.INT4, 128)
    assert float(kv[0, 1, 0, 70]) == 7 * 65504 and float(vv[0, 0, 1, 3]) == 7 * 1023
    assert float(vv[0, 2, 2, 127]) == 7 * 1023 and torch.isfinite(vv).all()


# ----------------------------------------------------------------------------- decode

def check_paged(lens, *, hkv=4, q_len=1, window=0, sink=False, seed=5, positions=None, q_mul=1.0, max_seq_len=None,
                edit=None, call=None, rows=None):
    g, r = gen(seed), np.random.default_rng(seed)
    B = len(lens)
    table, pages = R.table_of(lens, r)
    k, v, _, _ = R.random_cache(R.INT4, pages, g, hkv)
    if edit:
        edit(k, v, table)
    q = torch.randn((B * q_len, 64, 192), generator=g, device="cuda").mul_(q_mul).bfloat16()
    sk = torch.randn(64, generator=g, device="cuda") if sink else None
    base = 1e7 if hkv == 4 else 1e4
    out, lse = (call or M.mimo_attn_decode)(
        q, R.i32(lens), max_seq_len=max_seq_len or max(lens), num_kv_heads=hkv, rope_base=base, window=window,
        cache_kind=PAGED, k_cache=k, v_cache=v, block_table=table, num_pages=pages, sink=sk,
        cache_dtype=M.MIMO_DTYPE_INT4, **({} if q_len == 1 else dict(q_len=q_len)),
        **({} if positions is None else dict(positions=R.i32(positions))))
    assert M.status_poll() == 0
    for s in rows if rows is not None else range(B):
        n = lens[s]
        kv = R.slots_of(k[table[s][:-(-n // 128)].long()], R.INT4, 192).transpose(0, 1).flatten(1, 2)[:, :n]
        vv = R.slots_of(v[table[s][:-(-n // 128)].long()], R.INT4, 128).transpose(0, 1).flatten(1, 2)[:, :n]
        me = torch.arange(n - q_len, n, device="cuda")
        pos = None if positions is None else me - (n - 1) + positions[s]
        sl = slice(s * q_len, (s + 1) * q_len)
        R.Row(q[sl], kv, vv, torch.arange(n, device="cuda"), me, base, pos=pos, window=window,
              sink=sk).check(out[sl], lse[sl], f"sequence {s} of {n}")
    return out, lse


@gpu
@pytest.mark.parametrize("lens", [[1], [31, 32, 33], [127, 128, 129, 255, 256, 257], [1, 500, 4000, 64, 2, 9000, 300]])
@pytest.mark.parametrize("q_len", [1, 2, 3, 4, 5, 8])
def test_decode_paged(lens, q_len):
    check_paged([max(x, q_len) for x in lens], q_len=q_len, seed=q_len)


@gpu
@pytest.mark.parametrize("q_len", [1, 2, 5, 8])
@pytest.mark.parametrize("window", [0, 1, 130, 700])
def test_decode_paged_8_heads_window_sink(q_len, window):
    check_paged([8, 129, 1500, 2049], hkv=8, q_len=q_len, window=window, sink=True, seed=20 + q_len)


@gpu
def test_decode_long_and_many():
    check_paged([70001], seed=30)
    check_paged([40000, 8], q_len=8, seed=31)
    check_paged([int(x) for x in np.random.default_rng(1).integers(1, 900, 300)], seed=32, rows=range(0, 300, 7))


@gpu
def test_decode_more_sequences_than_one_launch():
    lens = [int(x) for x in np.random.default_rng(2).integers(1, 600, 1100)]
    check_paged(lens, seed=33, rows=[0, 5, 1023, 1024, 1025, 1099])


@gpu
@pytest.mark.parametrize("q_len", [1, 2, 6])
def test_decode_positions(q_len):
    check_paged([200, 1000, 9], q_len=q_len, seed=34, positions=[5000, 120000, 8])


@gpu
def test_decode_wide_logits_and_max_seq_len():
    """Logits so wide that the running maximum moves often; a max_seq_len far above the lengths."""
    check_paged([3000, 700], q_mul=8.0, seed=35, max_seq_len=3000)
    check_paged([3000, 700], seed=36, max_seq_len=3000)


@gpu
@pytest.mark.parametrize("q_len", [2, 3, 4, 6, 8])
def test_decode_drafts_wide_logits(q_len):
    """The references of every number of columns move, with the sums of the tiles before."""
    check_paged([3000, 700], q_mul=8.0, q_len=q_len, seed=39)


@gpu
def test_decode_drafts_long():
    check_paged([70001, 300], q_len=4, seed=45)


@gpu
@pytest.mark.parametrize("q_len", [1, 4, 8])
def test_decode_a_nan_query_row_is_alone(q_len):
    """A row of NaN: NaN in its output and log-sum-exp, every other row bit for bit as without it."""
    g, lens = gen(46), [900, 131]
    table, pages = R.table_of(lens, np.random.default_rng(46))
    k, v, _, _ = R.random_cache(R.INT4, pages, g)
    q = torch.randn((2 * q_len, 64, 192), generator=g, device="cuda").bfloat16()
    run = lambda x: M.mimo_attn_decode(x, R.i32(lens), max_seq_len=900, num_kv_heads=4, rope_base=1e7, window=0,
                                       cache_kind=PAGED, k_cache=k, v_cache=v, block_table=table, num_pages=pages,
                                       cache_dtype=M.MIMO_DTYPE_INT4, q_len=q_len)
    o1, l1 = run(q)
    bad = q.clone()
    bad[q_len, 37] = float("nan")
    o2, l2 = run(bad)
    assert torch.isnan(o2[q_len, 37]).all() and torch.isnan(l2[q_len, 37])
    o2[q_len, 37], l2[q_len, 37] = o1[q_len, 37], l1[q_len, 37]
    assert torch.equal(o1, o2) and torch.equal(l1, l2)
    M.status_poll()


@gpu
def test_decode_two_streams_and_two_graphs_at_once():
    """Calls that run at the same time, each with its workspace: the results of the calls alone."""
    g = gen(47)
    sets = []
    for i, lens in enumerate(([30000], [20000, 7, 4000])):
        table, pages = R.table_of(lens, np.random.default_rng(47 + i))
        k, v, _, _ = R.random_cache(R.INT4, pages, g)
        q = torch.randn((len(lens), 64, 192), generator=g, device="cuda").bfloat16()
        kw = dict(max_seq_len=max(lens), num_kv_heads=4, rope_base=1e7, window=0, cache_kind=PAGED, k_cache=k, v_cache=v,
                  block_table=table, num_pages=pages, cache_dtype=M.MIMO_DTYPE_INT4)
        sets.append((q, R.i32(lens), kw, M.mimo_attn_decode(q, R.i32(lens), **kw)))
    torch.cuda.synchronize()
    streams, got = [torch.cuda.Stream() for _ in sets], []
    for _ in range(3):
        for st, (q, lens, kw, _r) in zip(streams, sets):
            with torch.cuda.stream(st):
                got.append((M.mimo_attn_decode(q, lens, **kw), _r))
    torch.cuda.synchronize()
    graphs = []
    for q, lens, kw, ref in sets:
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            r = M.mimo_attn_decode(q, lens, **kw)
        graphs.append((graph, r, ref))
    for st, (graph, r, ref) in zip(streams, graphs):
        with torch.cuda.stream(st):
            graph.replay()
            graph.replay()
    torch.cuda.synchronize()
    for r, ref in got + [(r, ref) for _, r, ref in graphs]:
        assert torch.equal(r[0], ref[0]) and torch.equal(r[1], ref[1])
    assert M.status_poll() == 0


@gpu
def test_decode_ignores_what_lies_behind():
    """Slots from seq_lens on may hold anything: NaN and infinite scales change nothing."""
    def spoil(k, v, table):
        for c, codes, per in ((k, 96, 12), (v, 64, 8)):
            s = c[..., 128 * codes:].view(torch.half).view(c.shape[0], 4, 128, per // 2)
            page = int(table[0, 1])
            s[page, :, 40:] = float("nan")
            s[page, :, 41] = float("inf")
            c[page, :, 40 * codes:128 * codes] = 0xFF
    check_paged([168], seed=37, edit=spoil)
    check_paged([168], seed=37, q_len=4, edit=spoil)


@gpu
def test_decode_negative_and_extreme_scales():
    """Scales of either sign, and value scales over twelve powers of two within a head."""
    def scales(k, v, table):
        for c, codes, n in ((k, 96, 6), (v, 64, 4)):
            s = c[..., 128 * codes:].view(torch.half)
            s *= torch.where(torch.rand(s.shape, device="cuda", generator=gen(1)) < 0.5, -1.0, 1.0).half()
        s *= torch.exp2(torch.randint(-8, 5, s.shape, device="cuda", generator=gen(2)).float()).half()
    check_paged([1200, 77], seed=38, edit=scales)


@gpu
@pytest.mark.parametrize("ring, q_len, window", [(128, 1, 128), (144, 1, 129), (144, 4, 128), (512, 8, 505), (160, 3, 20)])
@pytest.mark.parametrize("hkv", [8, 4])
def test_decode_ring(ring, q_len, window, hkv):
    g = gen(40 + ring)
    ctx = [q_len, 17 + q_len, ring - 1, ring, ring + 1, 3 * ring + 37, 100003]
    B = len(ctx)
    k, v, _, _ = R.random_cache(R.INT4, B, g, hkv, ring)
    q = torch.randn((B * q_len, 64, 192), generator=g, device="cuda").bfloat16()
    sk = torch.randn(64, generator=g, device="cuda")
    # slots that no position has reached hold garbage
    for c, codes in ((k, 96), (v, 64)):
        c[..., ring * codes:].view(torch.half).view(B, hkv, ring, -1)[1, :, ctx[1]:] = float("nan")
    out, lse = M.mimo_attn_decode(q, R.i32(ctx), max_seq_len=max(ctx), num_kv_heads=hkv, rope_base=1e4, window=window,
                                  cache_kind=RING, k_cache=k, v_cache=v, sink=sk, cache_dtype=M.MIMO_DTYPE_INT4,
                                  ring_slots=ring, q_len=q_len)
    assert M.status_poll() == 0
    kv, vv = R.slots_of(k, R.INT4, 192), R.slots_of(v, R.INT4, 128)
    for s, n in enumerate(ctx):
        at = torch.arange(max(0, n - ring), n, device="cuda")
        sl = slice(s * q_len, (s + 1) * q_len)
        R.Row(q[sl], kv[s][:, at % ring], vv[s][:, at % ring], at, torch.arange(n - q_len, n, device="cuda"), 1e4,
              window=window, sink=sk).check(out[sl], lse[sl], f"ring {ring}, context {n}")


@gpu
@pytest.mark.parametrize("B", [74, 80, 160])
def test_decode_many_rings(B):
    """More rings than workers, as many as pairs of them, and numbers between."""
    g, r = gen(48), np.random.default_rng(48)
    ctx = [int(x) for x in r.integers(1, 700, B)]
    k, v, _, _ = R.random_cache(R.INT4, B, g, 8, 128)
    q = torch.randn((B, 64, 192), generator=g, device="cuda").bfloat16()
    out, lse = M.mimo_attn_decode(q, R.i32(ctx), max_seq_len=700, num_kv_heads=8, rope_base=1e4, window=128, cache_kind=RING,
                                  k_cache=k, v_cache=v, cache_dtype=M.MIMO_DTYPE_INT4)
    assert M.status_poll() == 0
    for s in range(0, B, 9):
        n = ctx[s]
        at = torch.arange(max(0, n - 128), n, device="cuda")
        kv, vv = R.slots_of(k[s:s + 1], R.INT4, 192)[0], R.slots_of(v[s:s + 1], R.INT4, 128)[0]
        R.Row(q[s:s + 1], kv[:, at % 128], vv[:, at % 128], at, torch.arange(n - 1, n, device="cuda"), 1e4,
              window=128).check(out[s:s + 1], lse[s:s + 1], f"ring {s}")


@gpu
def test_decode_noalloc_and_streams():
    """The no-alloc call on a big batch (its pieces are cut to the array), a second stream, and
    a captured call replayed on new contents."""
    def noalloc(q, lens, **kw):
        out = torch.empty((q.shape[0], 64, 128), dtype=torch.bfloat16, device="cuda")
        lse = torch.empty((q.shape[0], 64), device="cuda")
        return M.mimo_attn_decode_noalloc(q, lens, out=out, lse=lse, **kw)
    check_paged([5000] * 24, seed=50, call=noalloc, rows=[0, 23])
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())

    def on_side(*a, **kw):
        torch.cuda.synchronize()
        r = M.mimo_attn_decode(*a, stream=side, **kw)
        side.synchronize()
        return r
    check_paged([5000, 60], seed=51, call=on_side)

    def captured(q, lens, **kw):
        ws = torch.empty(M.decode_workspace_size(len(lens), kw["max_seq_len"], 4, 0, 1, M.MIMO_DTYPE_INT4),
                         dtype=torch.uint8, device="cuda")
        out = torch.zeros((q.shape[0], 64, 128), dtype=torch.bfloat16, device="cuda")
        lse = torch.zeros((q.shape[0], 64), device="cuda")
        q2, l2 = torch.zeros_like(q), torch.ones_like(lens)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            M.mimo_attn_decode(q2, l2, out=out, lse=lse, workspace=ws, **kw)
        graph.replay()
        q2.copy_(q)
        l2.copy_(lens)
        graph.replay()
        return out, lse
    check_paged([5000, 60, 1], seed=52, call=captured)


@gpu
@pytest.mark.parametrize("kind", [PAGED, RING])
def test_decode_kernel_events(kind):
    """The events around the decode kernel, the merge behind them."""
    ev = [torch.cuda.Event(enable_timing=True) for _ in range(2)]
    for e in ev:
        e.record()
    g = gen(49)
    q = torch.randn((1, 64, 192), generator=g, device="cuda").bfloat16()
    if kind == PAGED:
        table, pages = R.table_of([5000], np.random.default_rng(49))
        k, v, _, _ = R.random_cache(R.INT4, pages, g)
        kw = dict(num_kv_heads=4, window=0, block_table=table, num_pages=pages)
    else:
        k, v, _, _ = R.random_cache(R.INT4, 1, g, 8, 128)
        kw = dict(num_kv_heads=8, window=128)
    run = lambda **e: M.mimo_attn_decode(q, R.i32([5000]), max_seq_len=5000, rope_base=1e6, cache_kind=kind, k_cache=k,
                                         v_cache=v, cache_dtype=M.MIMO_DTYPE_INT4, **kw, **e)
    a, b = run(), run(kernel_events=ev)
    torch.cuda.synchronize()
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
    assert 0 < ev[0].elapsed_time(ev[1]) < 50


@gpu
def test_decode_repeats_bit_for_bit():
    a = check_paged([9000, 20, 700], seed=53)
    b = check_paged([9000, 20, 700], seed=53)
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


@gpu
def test_decode_bad_lengths_and_pages_are_reported():
    g = gen(54)
    k, v, _, _ = R.random_cache(R.INT4, 4, g)
    q = torch.randn((2, 64, 192), generator=g, device="cuda").bfloat16()
    kw = dict(num_kv_heads=4, rope_base=1e7, window=0, cache_kind=PAGED, k_cache=k, v_cache=v, num_pages=4,
              cache_dtype=M.MIMO_DTYPE_INT4)
    good = R.i32([[0, 1], [2, 3]])
    for lens, table, msl in (([0, 200], good, 256), ([200, 257], good, 256), ([200, 200], R.i32([[0, 1], [2, 4]]), 256),
                             ([200, 200], R.i32([[0, -1], [2, 3]]), 256)):
        M.mimo_attn_decode(q, R.i32(lens), max_seq_len=msl, block_table=table, **kw)
        assert M.status_poll() == M.MIMO_STATUS_BAD_INDEX
    q[0, 3, 100] = 20000.0
    M.mimo_attn_decode(q, R.i32([200, 200]), max_seq_len=256, block_table=good, **kw)
    assert M.status_poll() == M.MIMO_STATUS_RANGE


@gpu
def test_append_then_decode():
    """As served: a prompt's rows appended, then steps of append + decode, each against float64
    on the cache's own contents."""
    g, r = gen(60), np.random.default_rng(60)
    lens, steps = [1, 300, 129], 4
    full = [n + steps for n in lens]
    table, pages = R.table_of(full, r)
    k, v = M.empty_int4_cache(pages, 4)
    kw = dict(cache_kind=PAGED, block_table=table, num_pages=pages)
    n = sum(lens)
    kn, vn = (torch.randn((n, 4, d), generator=g, device="cuda").bfloat16() for d in (192, 128))
    _append(kn, vn, R.i32(np.concatenate([np.arange(x) for x in lens])), R.i32(np.repeat(np.arange(3), lens)), k, v, 1e7,
            num_seqs=3, **kw)
    for i in range(steps):
        kn, vn = (torch.randn((3, 4, d), generator=g, device="cuda").bfloat16() for d in (192, 128))
        _append(kn, vn, R.i32([x + i for x in lens]), R.i32([0, 1, 2]), k, v, 1e7, num_seqs=3, **kw)
        q = torch.randn((3, 64, 192), generator=g, device="cuda").bfloat16()
        now = [x + i + 1 for x in lens]
        out, lse = M.mimo_attn_decode(q, R.i32(now), max_seq_len=max(now), num_kv_heads=4, rope_base=1e7, window=0,
                                      k_cache=k, v_cache=v, cache_dtype=M.MIMO_DTYPE_INT4, **kw)
        kv, vv = R.slots_of(k, R.INT4, 192), R.slots_of(v, R.INT4, 128)
        for s, m in enumerate(now):
            R.Row(q[s:s + 1], R.pages_of(kv, table[s], m), R.pages_of(vv, table[s], m), torch.arange(m, device="cuda"),
                  torch.tensor([m - 1], device="cuda"), 1e7).check(out[s:s + 1], lse[s:s + 1], f"step {i}")
    assert M.status_poll() == 0


@gpu
@pytest.mark.parametrize("q_len", [1, 2, 4, 8])
def test_decode_one_dominant_key_over_a_flat_tail(q_len):
    """A first key that takes nearly all the weight and has a zero value (what trained heads do), over
    131000 keys whose weights are 2^20 to 2^25.5 below it, by head, and whose values share a sign: the
    output is the tail's alone.  (In fp16 without a bias, weights below 2^-25 are zero.)"""
    g, n = gen(70), 131001
    table, pages = R.table_of([n], np.random.default_rng(70))
    kc = torch.full((pages, 4, 128, 192), 8, dtype=torch.uint8, device="cuda")  # zeros: every tail logit is 0
    vc = torch.randint(9, 16, (pages, 4, 128, 128), generator=g, device="cuda", dtype=torch.uint8)
    first = int(table[0, 0])
    kc[first, :, 0, 100] = 15
    vc[first, :, 0] = 8
    k = R.int4_block(kc, torch.ones((pages, 4, 128, 6), device="cuda"))
    v = R.int4_block(vc, torch.rand((pages, 4, 128, 4), generator=g, device="cuda") * 0.3 + 0.05)
    del kc, vc
    q = torch.zeros((q_len, 64, 192), device="cuda", dtype=torch.bfloat16)
    for i in range(q_len):  # the logit of key 0 in powers of two: 20 .. 25.5, spread differently in every draft
        x = 20 + 5.5 * ((torch.arange(64, device="cuda") * 7 + i) % 64) / 63
        q[i, :, 100] = (x * np.log(2.0) / (7 * R.SCALE)).bfloat16()
    out, lse = M.mimo_attn_decode(q, R.i32([n]), max_seq_len=n, num_kv_heads=4, rope_base=1e7, window=0, cache_kind=PAGED,
                                  k_cache=k, v_cache=v, block_table=table, num_pages=pages, cache_dtype=M.MIMO_DTYPE_INT4,
                                  q_len=q_len)
    assert M.status_poll() == 0
    kv, vv = (R.pages_of(R.slots_of(c, R.INT4, d), table[0], n) for c, d in ((k, 192), (v, 128)))
    R.Row(q, kv, vv, torch.arange(n, device="cuda"), torch.arange(n - q_len, n, device="cuda"), 1e7).check(out, lse)


@gpu
def test_memory_made_for_another_stream(monkeypatch):
    """What a call with stream= allocates belongs to that stream: no block of it is handed out on the
    current stream while the call may still run, and none that the current stream may still use is
    taken for it."""
    g = gen(71)
    side, made = torch.cuda.Stream(), []
    table, pages = R.table_of([5000], np.random.default_rng(71))
    k, v, _, _ = R.random_cache(R.INT4, pages, g)
    q = torch.randn((1, 64, 192), generator=g, device="cuda").bfloat16()
    lens = R.i32([5000])
    kw = dict(max_seq_len=5000, num_kv_heads=4, rope_base=1e7, window=0, cache_kind=PAGED, k_cache=k, v_cache=v,
              block_table=table, num_pages=pages, cache_dtype=M.MIMO_DTYPE_INT4)
    want = M.mimo_attn_decode(q, lens, **kw)
    need = M.decode_workspace_size(1, 5000, 4, 0, 1, M.MIMO_DTYPE_INT4)
    scores = torch.rand((1, 4, 5000), generator=g, device="cuda")
    picked = M.mimo_kv_select(scores, lens, max_seq_len=5000, keep=300)
    torch.cuda.synchronize()
    sizes = [need, q.numel() // 192 * 128 * 2, 64 * 4, 300 * 4 * 4]

    def current_blocks():  # blocks that the current stream has just given back
        x = [torch.empty(s, dtype=torch.uint8, device="cuda") for s in sizes]
        return {t.data_ptr() for t in x}
    plain, new_empty = torch.empty, torch.Tensor.new_empty

    def note(f):
        def wrapped(*a, **k):
            t = f(*a, **k)
            made.append(t.data_ptr())
            return t
        return wrapped
    for stream in (side, side.cuda_stream):
        free = current_blocks()
        made.clear()
        with torch.cuda.stream(side):
            torch.cuda._sleep(50_000_000)  # some 25 ms
        with monkeypatch.context() as m:
            m.setattr(torch, "empty", note(plain))
            m.setattr(torch.Tensor, "new_empty", note(new_empty))
            got = M.mimo_attn_decode(q, lens, stream=stream, **kw)
            sel = M.mimo_kv_select(scores, lens, max_seq_len=5000, keep=300, stream=stream)
        assert len(made) >= 6 and not free & set(made)
        assert not current_blocks() & set(made)
        side.synchronize()
        for a, b in zip(got + sel, want + picked):
            assert torch.equal(a, b)
    assert M.status_poll() == 0


@pytest.mark.parametrize("hkv", [4, 8])
def test_workspace_size_never_shrinks(hkv):
    """A buffer for the largest batch and context serves every smaller one."""
    size = M.lib().mimo_attn_decode_int4_workspace_size
    for q_len in (1, 2, 4, 8):
        for n in (257, 300, 512, 513, 700, 1000, 1024, 1025, 5000, 100000):
            over_batch = [size(b, q_len, n, hkv, 0, PAGED) for b in list(range(1, 160)) + [500, 1023, 1024, 1025, 5000]]
            assert over_batch == sorted(over_batch) and over_batch[0] > 0
        for b in (1, 7, 24, 25, 64, 300):
            over_keys = [size(b, q_len, n, hkv, 0, PAGED) for n in range(q_len, 3000, 7)]
            assert over_keys == sorted(over_keys)
    # units of up to 512 keys are never cut: no pieces to hold
    assert size(64, 1, 512, 4, 0, PAGED) < 1024


@gpu
@pytest.mark.parametrize("q_len", [1, 4])
def test_decode_with_a_buffer_for_a_larger_batch(q_len):
    """One buffer, sized for the largest batch, through batches on either side of whole and cut units."""
    ws = torch.empty(M.decode_workspace_size(48, 1000, 4, 0, q_len, M.MIMO_DTYPE_INT4), dtype=torch.uint8, device="cuda")
    for B in (48, 25, 24, 13, 12, 1):
        lens = [1000] + [int(x) for x in np.random.default_rng(B).integers(q_len, 1001, B - 1)]  # (8 pages)
        check_paged(lens, q_len=q_len, seed=72, max_seq_len=1000, rows=[0, B - 1],
                    call=lambda *a, **kw: M.mimo_attn_decode(*a, workspace=ws, **kw))


@gpu
def test_decode_ring_reports_lengths_above_the_bound():
    """As over pages; the rows are those of a call with a bound that holds."""
    g = gen(55)
    k, v, _, _ = R.random_cache(R.INT4, 3, g, 8, 128)
    q = torch.randn((3, 64, 192), generator=g, device="cuda").bfloat16()
    run = lambda n: M.mimo_attn_decode(q, R.i32([50, 301, 200]), max_seq_len=n, num_kv_heads=8, rope_base=1e4, window=128,
                                       cache_kind=RING, k_cache=k, v_cache=v, cache_dtype=M.MIMO_DTYPE_INT4)
    a = run(301)
    assert M.status_poll() == 0
    b = run(300)
    assert M.status_poll() == M.MIMO_STATUS_BAD_INDEX
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


@gpu
@pytest.mark.parametrize("fmt", [R.BF16, R.INT4])
def test_decode_noalloc_drafts_and_positions(fmt):
    """The call that allocates nothing takes what the other takes: the same rows."""
    g, r = gen(73), np.random.default_rng(73)
    lens, pos, q_len = [300, 1200], [9000, 1199], 3
    table, pages = R.table_of(lens, r)
    k, v, _, _ = R.random_cache(fmt, pages, g)
    q = torch.randn((2 * q_len, 64, 192), generator=g, device="cuda").bfloat16()
    for p in (None, R.i32(pos)):
        kw = dict(max_seq_len=1200, num_kv_heads=4, rope_base=1e7, window=0, cache_kind=PAGED, k_cache=k, v_cache=v,
                  block_table=table, num_pages=pages, cache_dtype=fmt, q_len=q_len, positions=p)
        out, lse = torch.empty((6, 64, 128), dtype=torch.bfloat16, device="cuda"), torch.empty((6, 64), device="cuda")
        M.mimo_attn_decode_noalloc(q, R.i32(lens), out=out, lse=lse, **kw)
        want = M.mimo_attn_decode(q, R.i32(lens), **kw)
        assert torch.equal(out, want[0]) and torch.equal(lse, want[1])
    assert M.status_poll() == 0


@gpu
@pytest.mark.parametrize("tokens, calls", [(20000, 2), (400, 60)])
@pytest.mark.parametrize("base, hkv", [(1e7, 4), (1e4, 8)])
def test_append_codes_of_the_exact_rotation(tokens, calls, base, hkv):
    """Every code and scale is the rule's on the rotation in 64 bits, also where a quotient or a scale lies
    next to a border (a rotation in fp32 moves some tens of 5 million codes)."""
    g, r = gen(80), np.random.default_rng(80)
    blocks = -(-tokens // 128)
    table = R.i32(r.permutation(blocks)[None])
    seq, slots = torch.zeros(tokens, dtype=torch.int32, device="cuda"), R.i32(np.arange(tokens))

    def rule(x):
        x = x.unflatten(-1, (-1, 32))
        s = (x.abs().amax(-1) / 7).float().half().double()[..., None]
        n = torch.where(s > 0, torch.round(x / s).clamp(-7, 7), torch.zeros_like(x))
        return (n * s).flatten(-2)
    for _ in range(calls):
        kn = torch.randn((tokens, hkv, 192), generator=g, device="cuda").mul_(2).bfloat16()
        vn = torch.randn((tokens, hkv, 128), generator=g, device="cuda").bfloat16()
        pos = R.i32(r.integers(0, 131072, tokens))
        k, v = M.empty_int4_cache(blocks, hkv)
        _append(kn, vn, pos, seq, k, v, base, cache_kind=PAGED, num_seqs=1, block_table=table, num_pages=blocks, slots=slots)
        got = R.pages_of(R.slots_of(k, R.INT4, 192), table[0], tokens).transpose(0, 1)
        assert torch.equal(got, rule(R.rotate(kn, pos, base)))
        got = R.pages_of(R.slots_of(v, R.INT4, 128), table[0], tokens).transpose(0, 1)
        assert torch.equal(got, rule(vn.double()))
    assert M.status_poll() == 0


@gpu
def test_append_not_finite_beside_other_groups():
    """NaN and infinities in a key: +-7 of their group as the rule says, whatever the words beside them."""
    g = gen(81)
    n = 3000
    kn = torch.randn((n, 4, 192), generator=g, device="cuda").bfloat16()
    vn = torch.randn((n, 4, 128), generator=g, device="cuda").bfloat16()
    kn[::3, 1, 5], kn[1::3, 2, 40], kn[2::3, 0, 100] = float("inf"), float("nan"), -float("inf")
    k, v = M.empty_int4_cache(24, 4)
    pos = R.i32(np.arange(n))
    _append(kn, vn, pos, torch.zeros_like(pos), k, v, 1e7, cache_kind=PAGED, num_seqs=1, block_table=R.i32(np.arange(24)[None]),
            num_pages=24)
    assert M.status_poll() == M.MIMO_STATUS_RANGE
    got = R.pages_of(R.slots_of(k, R.INT4, 192), R.i32(np.arange(24)), n).transpose(0, 1)
    assert torch.isfinite(got).all()
    assert (got[2::3, 0, 100] == -7 * 65504).all() and (got[2::3, 0, 96:100] == 0).all()
    # (dims 5 and 37, 40 and 8 turn together; a NaN takes no part in its group's scale)
    want = R.rotate(kn, pos, 1e7)
    clean = torch.isfinite(want.unflatten(-1, (-1, 32))).all(-1)
    ref = want.unflatten(-1, (-1, 32))
    s = (ref.abs().amax(-1) / 7).float().half().double()[..., None]
    ref = torch.round(ref / s).clamp(-7, 7) * s
    assert torch.equal(got.unflatten(-1, (-1, 32))[clean], ref[clean])
    bad = ~torch.isfinite(want)
    assert bad.any() and (got[bad] != 0).all()
