"""Eviction from a paged cache: accumulated attention weights, the selection of slots, the gather
into other pages, and the calls together, against float64; refusals on the CPU."""
import ctypes as C

import numpy as np
import pytest
import torch

import global_attention_attn_b200 as M
from tests import cache_ref as R

gpu = pytest.mark.gpu
BF16, E4M3, INT4 = R.BF16, R.E4M3, R.INT4
PAGED = M.MIMO_CACHE_PAGED


def gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


# ----------------------------------------------------------------------------- refusals (host)

P = 1 << 20  # an address that is never read


def _weights(**kw):
    a = M.MimoWeightsArgs()
    a.layer = M.make_layer(kw.pop("hkv", 4), 1e7, kw.pop("window", 0))
    a.batch, a.q_len, a.max_seq_len, a.score_stride, a.max_pages, a.num_pages = 2, 1, 300, 384, 3, 6
    a.q = a.lse = a.seq_lens = a.k_cache = a.block_table = a.scores = P
    for k, v in kw.items():
        setattr(a, k, v)
    return M.lib().mimo_attn_weights(C.byref(a), None)


@pytest.mark.parametrize("kw", [dict(window=128), dict(q_len=9), dict(max_seq_len=400), dict(score_stride=299),
                                dict(lse=None), dict(scores=P + 4), dict(positions=P + 4), dict(cache_dtype=5),
                                dict(cache_dtype=E4M3), dict(cache_dtype=INT4, k_dequant=P), dict(max_seq_len=0),
                                dict(batch=-1)])
def test_weights_refusals(kw):
    assert _weights(**kw) == M.MIMO_ERR_INVALID_ARG
    assert "mimo_attn_weights" in M.lib().mimo_last_error().decode()


def _select(**kw):
    a = M.MimoSelectArgs()
    a.num_seqs, a.num_kv_heads, a.score_stride, a.max_seq_len, a.keep, a.recent, a.first = 2, 4, 300, 300, 64, 8, 4
    a.scores = a.seq_lens = a.idx = a.counts = a.scores_out = P
    for k, v in kw.items():
        setattr(a, k, v)
    return M.lib().mimo_kv_select(C.byref(a), None)


@pytest.mark.parametrize("kw", [dict(keep=0), dict(recent=61), dict(recent=-1), dict(first=-1), dict(score_stride=299),
                                dict(max_seq_len=M.MIMO_SELECT_MAX_SLOTS + 1, score_stride=1 << 20), dict(idx=None),
                                dict(counts=None), dict(scores=P + 4), dict(max_seq_len=0)])
def test_select_refusals(kw):
    assert _select(**kw) == M.MIMO_ERR_INVALID_ARG
    assert "mimo_kv_select" in M.lib().mimo_last_error().decode()


def _gather(**kw):
    a = M.MimoGatherArgs()
    a.num_seqs, a.num_kv_heads, a.max_pages_src, a.num_pages_src, a.max_pages_dst, a.num_pages_dst = 2, 4, 3, 6, 1, 2
    a.k_src = a.v_src = a.block_table_src = a.k_dst = a.v_dst = a.block_table_dst = a.counts = a.idx = P
    a.idx_stride, a.max_count, a.cache_dtype, a.out_dtype = 128, 128, BF16, BF16
    for k, v in kw.items():
        setattr(a, k, v)
    return M.lib().mimo_kv_gather(C.byref(a), None)


@pytest.mark.parametrize("kw", [dict(max_count=129), dict(idx_stride=127), dict(out_dtype=E4M3), dict(cache_dtype=E4M3),
                                dict(cache_dtype=INT4, k_dequant=P), dict(cache_dtype=INT4, out_dtype=E4M3),
                                dict(counts=None), dict(k_dst=P + 8), dict(max_pages_dst=0), dict(num_seqs=70000)])
def test_gather_refusals(kw):
    assert _gather(**kw) == M.MIMO_ERR_INVALID_ARG
    assert "mimo_kv_gather" in M.lib().mimo_last_error().decode()


def test_python_refusals(monkeypatch):
    """What the binding can see of a tensor: element sizes, shapes, the device."""
    s, n = torch.zeros((2, 4, 64)), torch.ones(2, dtype=torch.int32)
    for bad in (s.half(), s[:, :, ::2], s[0]):
        with pytest.raises(ValueError, match="scores"):
            M.mimo_kv_select(bad, n, max_seq_len=32, keep=8, stream=0)
        with pytest.raises(ValueError, match="scores"):
            M.mimo_attn_weights(torch.zeros((2, 64, 192), dtype=torch.bfloat16), torch.zeros((2, 64)), bad, n, max_seq_len=32,
                                num_kv_heads=4, rope_base=1e7, k_cache=s, block_table=n[:, None], num_pages=1, stream=0)
    for kw in (dict(idx=torch.zeros((2, 4, 7), dtype=torch.int32)), dict(idx=torch.zeros((2, 4, 8), dtype=torch.int64)),
               dict(counts=torch.zeros(3, dtype=torch.int32)), dict(scores_out=torch.zeros((2, 4, 8), dtype=torch.half))):
        with pytest.raises(ValueError, match=next(iter(kw))):
            M.mimo_kv_select(s, n, max_seq_len=64, keep=8, stream=0, **kw)
    with pytest.raises(ValueError, match="idx"):
        M.mimo_kv_gather(s, s, n[:, None], s, s, n[:, None], n, num_kv_heads=4, num_pages=1, num_pages_out=1,
                         idx=torch.zeros((2, 4, 8), dtype=torch.int64), stream=0)
    other = type("T", (), dict(is_cuda=True, device=torch.device("cuda", 1)))()
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)
    with pytest.raises(ValueError, match="current device"):
        M._stream(None, other)


def test_unsupported_heads():
    assert _weights(hkv=2) == _select(num_kv_heads=2) == _gather(num_kv_heads=16) == M.MIMO_ERR_UNSUPPORTED


# ----------------------------------------------------------------------------- accumulated weights

def check_weights(lens, fmt, *, hkv=4, q_len=1, seed=1, positions=None, edit=None, rows=None):
    g, r = gen(seed), np.random.default_rng(seed)
    B, base = len(lens), 1e7
    table, pages = R.table_of(lens, r)
    k, _, kd, _ = R.random_cache(fmt, pages, g, hkv)
    if edit:
        edit(k, table)
    q = torch.randn((B * q_len, 64, 192), generator=g, device="cuda").bfloat16()
    stride = (max(lens) + 130) // 4 * 4
    scores = torch.rand((B, hkv, stride), generator=g, device="cuda")
    before = scores.clone()
    ref = []
    lse = torch.zeros((B * q_len, 64), device="cuda")
    for s, n in enumerate(lens):
        kv = R.slots_of(k[table[s][:-(-n // 128)].long()], fmt, 192, kd).transpose(0, 1).flatten(1, 2)[:, :n]
        me = torch.arange(n - q_len, n, device="cuda")
        row = R.Row(q[s * q_len:(s + 1) * q_len], kv, None, torch.arange(n, device="cuda"), me, base,
                    pos=None if positions is None else me - (n - 1) + positions[s])
        lse[s * q_len:(s + 1) * q_len] = row.lse
        # the probabilities that the float32 lse stands for, and the size of their logits
        got = row.p * torch.exp(row.lse - lse[s * q_len:(s + 1) * q_len].double()).view(q_len, hkv, -1, 1)
        ref.append((got.sum((0, 2)), float(row.p.clamp(min=1e-300).log().add(row.lse.view(q_len, hkv, -1, 1)).abs()
                                            [row.p > 0].max())))
    out = M.mimo_attn_weights(q, lse, scores, R.i32(lens), max_seq_len=max(lens), num_kv_heads=hkv, rope_base=base,
                              k_cache=k, block_table=table, num_pages=pages, cache_dtype=fmt, k_dequant=kd, q_len=q_len,
                              positions=None if positions is None else R.i32(positions))
    assert out is scores and M.status_poll() == 0
    for s, n in enumerate(lens):
        if rows is not None and s not in rows:
            continue
        assert torch.equal(scores[s, :, n:], before[s, :, n:])
        add, zmax = ref[s]
        err = (scores[s, :, :n].double() - before[s, :, :n].double() - add).abs()
        # A probability exp(z - lse): fp32 sums of 192 products lose up to 2^-22 of their largest
        # partial sum at each of 16 steps (|z| <= zmax; partial sums up to about 4 zmax), z - lse
        # half a step of itself, the two-term query 2^-22 of z: 2^-17 (1 + zmax) covers them;
        # the stored sum half a step of itself
        tol = 2.0 ** -17 * (1 + zmax) * add + 2.0 ** -23 * (before[s, :, :n].double() + add) + 1e-9
        worst = float((err / tol).max())
        assert worst <= 1, f"sequence {s} of {n}: off by {worst:.3g} of its bound"
    return scores


@gpu
@pytest.mark.parametrize("fmt", [BF16, E4M3, INT4])
@pytest.mark.parametrize("q_len", [1, 2, 5, 8])
@pytest.mark.parametrize("hkv", [4, 8])
def test_weights(fmt, q_len, hkv):
    check_weights([q_len, 31 + q_len, 128, 129, 700, 5000], fmt, q_len=q_len, hkv=hkv, seed=q_len)


@gpu
@pytest.mark.parametrize("fmt", [BF16, E4M3, INT4])
def test_weights_long_many_positions(fmt):
    check_weights([60001], fmt, seed=20)
    check_weights([900, 130], fmt, seed=21, q_len=3, positions=[70000, 131])
    check_weights([int(x) for x in np.random.default_rng(1).integers(1, 300, 1030)], fmt, seed=22, rows=[0, 1023, 1024, 1029])


@gpu
@pytest.mark.parametrize("fmt", [BF16, INT4])
def test_weights_ignore_what_lies_behind(fmt):
    def spoil(k, table):
        page = int(table[0, 1])
        if fmt == BF16:
            k[page, 40:] = float("nan")
        else:
            k[page, :, 128 * 96:].view(torch.half).view(4, 128, 6)[:, 40:] = float("nan")
    check_weights([168], fmt, seed=23, edit=spoil)


@gpu
def test_weights_rows_without_a_sum_add_nothing():
    g = gen(24)
    k, _, _, _ = R.random_cache(BF16, 2, g)
    q = torch.randn((2, 64, 192), generator=g, device="cuda").bfloat16()
    lse = torch.full((2, 64), float("-inf"), device="cuda")
    lse[1, ::2], lse[1, 1::2] = float("inf"), float("nan")
    scores = torch.rand((2, 4, 128), generator=g, device="cuda")
    before = scores.clone()
    kw = dict(max_seq_len=100, num_kv_heads=4, rope_base=1e7, k_cache=k, num_pages=2)
    M.mimo_attn_weights(q, lse, scores, R.i32([100, 60]), block_table=R.i32([[0], [1]]), **kw)
    assert torch.equal(scores, before) and M.status_poll() == 0
    # lengths and pages outside their bounds are reported
    for lens, table in (([0, 60], [[0], [1]]), ([101, 60], [[0], [1]]), ([100, 60], [[0], [2]]), ([100, 60], [[-1], [1]])):
        M.mimo_attn_weights(q, lse, scores, R.i32(lens), block_table=R.i32(table), **kw)
        assert M.status_poll() == M.MIMO_STATUS_BAD_INDEX


@gpu
@pytest.mark.parametrize("fmt", [BF16, E4M3, INT4])
def test_weights_of_a_decode_call_sum_to_its_heads(fmt):
    """With decode's own lse, and a graph replayed three times: every KV head's weights sum to the
    16 heads (3 times), up to what decode's fp16 query moves its lse by."""
    g, r = gen(25), np.random.default_rng(25)
    lens = [1, 1000, 3001]
    table, pages = R.table_of(lens, r)
    k, v, kd, vd = R.random_cache(fmt, pages, g)
    q = torch.randn((3, 64, 192), generator=g, device="cuda").bfloat16()
    kw = dict(max_seq_len=3001, num_kv_heads=4, rope_base=1e7, k_cache=k, block_table=table, num_pages=pages, cache_dtype=fmt,
              k_dequant=kd)
    lens = R.i32(lens)
    _, lse = M.mimo_attn_decode(q, lens, window=0, cache_kind=PAGED, v_cache=v, v_dequant=vd, **kw)
    scores = torch.zeros((3, 4, 3004), device="cuda")
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        M.mimo_attn_weights(q, lse, scores, lens, **kw)
    for _ in range(3):
        graph.replay()
    assert M.status_poll() == 0
    assert float((scores.double().sum(-1) - 48).abs().max()) < 48 * 2e-3


# ----------------------------------------------------------------------------- selection

def select_ref(scores, lens, keep, recent, first):
    n, h, _ = scores.shape
    x = torch.nan_to_num(scores, nan=-float("inf"), posinf=float("inf"), neginf=-float("inf")).cpu().numpy()
    idx = np.full((n, h, keep), -1, np.int32)
    for s in range(n):
        t = np.arange(lens[s])
        forced = (t < first) | (t >= lens[s] - recent)
        for g in range(h):
            row = x[s, g, :lens[s]].astype(np.float64) + 0.0
            kept = np.sort(np.lexsort((t, -row, ~forced))[:keep])
            idx[s, g, :len(kept)] = kept
    return torch.from_numpy(idx)


def check_select(scores, lens, keep, recent=0, first=0, **kw):
    idx, counts, vals = M.mimo_kv_select(scores, R.i32(lens), max_seq_len=max(max(lens), 1), keep=keep, recent=recent,
                                         first=first, **kw)
    torch.cuda.synchronize()
    want = select_ref(scores, lens, keep, recent, first)
    assert torch.equal(idx.cpu(), want)
    assert counts.tolist() == [min(x, keep) for x in lens]
    w = want.long().cuda()
    sel = scores.gather(-1, w.clamp(min=0))
    sel = torch.where(w >= 0, sel, torch.zeros_like(sel))
    assert torch.equal(vals.view(torch.int32), sel.view(torch.int32))
    assert M.status_poll() == 0


@gpu
@pytest.mark.parametrize("hkv", [4, 8])
@pytest.mark.parametrize("lens, keep, recent, first", [
    ([1], 1, 0, 0), ([1, 2, 3], 2, 1, 1), ([0, 5, 64], 64, 3, 4), ([63, 64, 65, 66], 64, 64, 0), ([100, 33], 20, 0, 20),
    ([4096, 4097, 5000], 1000, 100, 4), ([20000, 3, 12345], 8191, 0, 0), ([40000], 39999, 7, 7), ([70000, 69999], 17, 16, 0),
])
def test_select(lens, keep, recent, first, hkv):
    g = gen(keep)
    scores = torch.randn((len(lens), hkv, max(lens) + 3), generator=g, device="cuda")
    check_select(scores, lens, keep, recent, first)


@gpu
@pytest.mark.parametrize("B, lo, hi, keep, recent", [(40, 5000, 9000, 2000, 64), (16, 70000, 140000, 9000, 0), (20, 1, 66000, 3000, 9),
                                                     (5, 300000, 390000, 20000, 128)])
def test_select_many_rows(B, lo, hi, keep, recent):
    """More rows than one round of CTAs holds; half of the scores are equal."""
    g = gen(B)
    lens = [int(x) for x in np.random.default_rng(B).integers(lo, hi + 1, B)]
    scores = torch.randn((B, 8, max(lens)), generator=g, device="cuda")
    scores = torch.where(torch.rand(scores.shape, generator=g, device="cuda") < 0.5, torch.full_like(scores, 0.5), scores)
    check_select(scores, lens, keep, recent, 4)
    scores[scores == 0.5] = 0.0
    check_select(scores, lens, lo // 2 + 5 + recent, recent, 4)


@gpu
@pytest.mark.parametrize("n", [500, 9000, 50001])
def test_select_ties_and_specials(n):
    g = gen(n)
    x = torch.rand((2, 4, n), generator=g, device="cuda")
    few = (x * 5).floor() / 4 - 0.5                       # five values, zero among them
    check_select(few, [n, n - 7], n // 3, 5, 3)
    check_select(torch.zeros_like(x), [n, n // 2 + 1], n // 2, 0, 1)
    odd = torch.where(x < 0.2, float("nan"), torch.where(x < 0.4, -float("inf"), torch.where(x < 0.5, float("inf"),
                      torch.where(x < 0.7, -0.0, torch.where(x < 0.9, 0.0, 1e-42)))))
    for keep in (n // 20, n // 5, n // 2, (9 * n) // 10):
        check_select(odd, [n, n - 1], keep, 2, 2)
    check_select(torch.exp(-60 * x), [n, n], n // 4, 0, 0)  # twenty-six orders of magnitude


@gpu
def test_select_largest_and_bad_lengths():
    n = M.MIMO_SELECT_MAX_SLOTS
    scores = torch.rand((1, 4, n), generator=gen(3), device="cuda")
    check_select(scores, [n], 16384, 1024, 4)
    out = M.mimo_kv_select(scores, R.i32([-3]), max_seq_len=100, keep=5)
    assert M.status_poll() == M.MIMO_STATUS_BAD_INDEX and int(out[1]) == 0 and (out[0] == -1).all()
    out = M.mimo_kv_select(scores, R.i32([101]), max_seq_len=100, keep=5)
    assert M.status_poll() == M.MIMO_STATUS_BAD_INDEX and int(out[0].max()) < 100


# ----------------------------------------------------------------------------- gather

def _empty(fmt, pages, hkv):
    if fmt == INT4:
        return M.empty_int4_cache(pages, hkv)
    dt = torch.uint8 if fmt == E4M3 else torch.bfloat16
    return tuple(torch.zeros((pages, 128, hkv, d), dtype=dt, device="cuda") for d in (192, 128))


def check_gather(lens, counts, src, dst, *, hkv=4, seed=1, identity=False):
    g, r = gen(seed), np.random.default_rng(seed)
    B = len(lens)
    table, pages = R.table_of(lens, r)
    k, v, kd, vd = R.random_cache(src, pages, g, hkv)
    out_table, out_pages = R.table_of(counts, r, spare=1)
    ko, vo = _empty(dst, out_pages, hkv)
    ko.view(torch.uint8).fill_(0x5A)
    vo.view(torch.uint8).fill_(0x5A)
    k0, v0 = ko.clone(), vo.clone()
    cap = max(counts) + 3
    idx = torch.full((B, hkv, cap), -1, dtype=torch.int32)
    for s in range(B):
        for h in range(hkv):
            pick = np.arange(counts[s]) if identity else np.sort(r.choice(lens[s], counts[s], replace=False))
            idx[s, h, :counts[s]] = torch.from_numpy(pick.astype(np.int32))
    M.mimo_kv_gather(k, v, table, ko, vo, out_table, R.i32(counts), num_kv_heads=hkv, num_pages=pages, num_pages_out=out_pages,
                     idx=None if identity else idx.cuda(), max_count=max(counts), cache_dtype=src, out_dtype=dst,
                     k_dequant=kd if src != dst else None, v_dequant=vd if src != dst else None)
    assert M.status_poll() == 0
    for cache, out, out0, dims, dq in ((k, ko, k0, 192, kd), (v, vo, v0, 128, vd)):
        a = R.slots_of(cache, src, dims, dq)
        b = R.slots_of(out, dst, dims, dq)
        b0 = R.slots_of(out0, dst, dims, dq)
        wrote = torch.zeros(b.shape[:3], dtype=torch.bool, device="cuda")
        for s in range(B):
            for h in range(hkv):
                j = torch.arange(counts[s], device="cuda")
                i = idx[s, h, :counts[s]].long().cuda()
                p, t = out_table[s][j // 128].long(), j % 128
                want = a[table[s][i // 128].long(), h, i % 128]
                got = b[p, h, t]
                wrote[p, h, t] = True
                if src != dst and dims == 192:
                    want = torch.cat([want[:, :64].half().double(), want[:, 64:].bfloat16().double()], -1)
                elif src != dst:
                    want = want.bfloat16().double()
                assert torch.equal(got, want)
        assert torch.equal(b[~wrote].nan_to_num(nan=7e7), b0[~wrote].nan_to_num(nan=7e7))


@gpu
@pytest.mark.parametrize("src, dst", [(BF16, BF16), (E4M3, E4M3), (INT4, INT4), (E4M3, BF16), (INT4, BF16)])
@pytest.mark.parametrize("hkv", [4, 8])
def test_gather(src, dst, hkv):
    check_gather([1, 200, 1000, 129], [1, 128, 300, 127], src, dst, hkv=hkv, seed=hkv)
    check_gather([300, 128], [300, 0], src, dst, hkv=hkv, identity=True)


@gpu
def test_gather_skips_and_reports():
    g = gen(9)
    k, v, _, _ = R.random_cache(BF16, 3, g)
    table, out = R.i32([[0, 1]]), R.i32([[1]])
    idx = torch.zeros((1, 4, 4), dtype=torch.int32, device="cuda")
    idx[0, 2, 1], idx[0, 3, 2] = 256, -1
    ko, vo = _empty(BF16, 2, 4)
    kw = dict(num_kv_heads=4, num_pages=3, num_pages_out=2)
    M.mimo_kv_gather(k, v, table, ko, vo, out, R.i32([4]), idx=idx, **kw)
    assert M.status_poll() == M.MIMO_STATUS_BAD_INDEX
    want = k[0, 0].expand(4, 4, 192).clone()
    want[1, 2] = 0
    want[2, 3] = 0
    assert torch.equal(ko[1, :4], want) and not ko[1, 4:].any() and not ko[0].any()
    for t_out, cnt in (([[2]], [4]), ([[-1]], [4]), ([[1]], [5])):
        M.mimo_kv_gather(k, v, table, ko, vo, R.i32(t_out), R.i32(cnt), idx=idx, **kw)
        assert M.status_poll() & M.MIMO_STATUS_BAD_INDEX


# ----------------------------------------------------------------------------- together

@gpu
@pytest.mark.parametrize("fmt", [BF16, E4M3, INT4])
def test_serving_with_eviction(fmt):
    """Prompts appended, steps of decode with accumulated weights, an eviction into fresh pages, and
    steps over the shorter cache, whose appends go to slots and whose queries keep their
    positions: every output against float64 on the cache's contents."""
    g, r = gen(70), np.random.default_rng(70)
    lens, keep, recent = [700, 90, 1300], 256, 32
    B, extra = len(lens), 3
    kd = torch.full((4,), 0.03, device="cuda") if fmt == E4M3 else None
    vd = torch.full((4,), 0.02, device="cuda") if fmt == E4M3 else None
    table, pages = R.table_of([n + extra for n in lens], r)
    k, v = _empty(fmt, pages, 4)
    scores = torch.zeros((B, 4, max(lens) + extra), device="cuda")
    fm = dict(cache_dtype=fmt, k_dequant=kd)

    def append(n, pos, seq, kc, vc, tab, np_, slots=None):
        kn, vn = (torch.randn((n, 4, d), generator=g, device="cuda").bfloat16() for d in (192, 128))
        M.mimo_kv_append(kn, vn, R.i32(pos), R.i32(seq), rope_base=1e7, cache_kind=PAGED, k_cache=kc, v_cache=vc, num_seqs=B,
                         block_table=tab, num_pages=np_, slots=None if slots is None else R.i32(slots), v_dequant=vd, **fm)

    def step(now, pos, kc, vc, tab, np_, what):
        q = torch.randn((B, 64, 192), generator=g, device="cuda").bfloat16()
        kw = dict(max_seq_len=max(now), num_kv_heads=4, rope_base=1e7, k_cache=kc, block_table=tab, num_pages=np_,
                  positions=R.i32(pos), **fm)
        out, lse = M.mimo_attn_decode(q, R.i32(now), window=0, cache_kind=PAGED, v_cache=vc, v_dequant=vd, **kw)
        kv, vv = R.slots_of(kc, fmt, 192, kd), R.slots_of(vc, fmt, 128, vd)
        for s, n in enumerate(now):
            R.Row(q[s:s + 1], R.pages_of(kv, tab[s], n), R.pages_of(vv, tab[s], n), torch.arange(n, device="cuda"),
                  torch.tensor([n - 1], device="cuda"), 1e7, pos=torch.tensor([pos[s]], device="cuda"),
                  p_step=2.0 ** -8 if fmt == BF16 else 2.0 ** -10).check(out[s:s + 1], lse[s:s + 1], what)
        return q, lse, kw

    append(sum(lens), np.concatenate([np.arange(n) for n in lens]), np.repeat(np.arange(B), lens), k, v, table, pages)
    for i in range(extra):
        append(B, [n + i for n in lens], [0, 1, 2], k, v, table, pages)
        now = [n + i + 1 for n in lens]
        q, lse, kw = step(now, [x - 1 for x in now], k, v, table, pages, f"step {i}")
        M.mimo_attn_weights(q, lse, scores, R.i32(now), **kw)
    now = [n + extra for n in lens]
    idx, counts, kept = M.mimo_kv_select(scores, R.i32(now), max_seq_len=max(now), keep=keep, recent=recent, first=4)
    table2, pages2 = R.table_of([min(n, keep) + extra for n in now], r)
    k2, v2 = _empty(fmt, pages2, 4)
    M.mimo_kv_gather(k, v, table, k2, v2, table2, counts, num_kv_heads=4, num_pages=pages, num_pages_out=pages2, idx=idx,
                     cache_dtype=fmt)
    assert counts.tolist() == [256, 93, 256]
    assert torch.equal(idx.cpu(), select_ref(scores, now, keep, recent, 4))
    a, b = R.slots_of(k, fmt, 192, kd), R.slots_of(k2, fmt, 192, kd)
    for s in range(B):
        m = int(counts[s])
        src = R.pages_of(a, table[s], now[s])
        got = R.pages_of(b, table2[s], m)
        assert torch.equal(got, torch.stack([src[h, idx[s, h, :m].long()] for h in range(4)]))
    for i in range(extra):
        at = [int(c) + i for c in counts]
        pos = [n + i for n in now]
        append(B, pos, [0, 1, 2], k2, v2, table2, pages2, slots=at)
        step([x + 1 for x in at], pos, k2, v2, table2, pages2, f"evicted step {i}")
    assert M.status_poll() == 0


@gpu
@pytest.mark.parametrize("fmt", [E4M3, INT4])
def test_prefill_over_a_widened_cache(fmt):
    """A prefix stored narrow, gathered into bf16 pages, and a chunk of queries prefilled over it."""
    g, r = gen(80), np.random.default_rng(80)
    n, new = 500, 37
    table, pages = R.table_of([n], r)
    k, v, kd, vd = R.random_cache(fmt, pages, g)
    table2, pages2 = R.table_of([n + new], r)
    k2, v2 = _empty(BF16, pages2, 4)
    M.mimo_kv_gather(k, v, table, k2, v2, table2, R.i32([n]), num_kv_heads=4, num_pages=pages, num_pages_out=pages2,
                     cache_dtype=fmt, out_dtype=BF16, k_dequant=kd, v_dequant=vd)
    kn, vn = (torch.randn((new, 4, d), generator=g, device="cuda").bfloat16() for d in (192, 128))
    M.mimo_kv_append(kn, vn, R.i32(np.arange(n, n + new)), R.i32([0] * new), rope_base=1e7, cache_kind=PAGED, k_cache=k2,
                     v_cache=v2, num_seqs=1, block_table=table2, num_pages=pages2)
    q = torch.randn((new, 64, 192), generator=g, device="cuda").bfloat16()
    out, lse = M.mimo_attn_prefill(q, None, None, R.i32([0, new]), None, num_kv_heads=4, rope_base=1e7, window=0,
                                   cache_lens=R.i32([n + new]), cache_kind=PAGED, k_cache=k2, v_cache=v2, block_table=table2,
                                   num_pages=pages2)
    kv, vv = (R.pages_of(R.slots_of(c, BF16, d), table2[0], n + new) for c, d in ((k2, 192), (v2, 128)))
    R.Row(q, kv, vv, torch.arange(n + new, device="cuda"), torch.arange(n, n + new, device="cuda"), 1e7,
          p_step=2.0 ** -8).check(out, lse, "prefill")
    assert M.status_poll() == 0


def test_new_struct_layouts_match_c(tmp_path):
    import os
    import subprocess
    header = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "include", "mimoattn.h")
    structs = {"mimo_weights_args": M.MimoWeightsArgs, "mimo_select_args": M.MimoSelectArgs,
               "mimo_gather_args": M.MimoGatherArgs}
    lines = ["#include <stdio.h>", "#include <stddef.h>", f'#include "{header}"', "int main(void) {",
             'printf("%d %d %d %d\\n", MIMO_DTYPE_INT4, MIMO_INT4_K_SLOT_BYTES, MIMO_INT4_V_SLOT_BYTES, MIMO_SELECT_MAX_SLOTS);']
    for c, py in structs.items():
        lines.append(f'printf("%zu\\n", sizeof({c}));')
        lines += [f'printf("%zu\\n", offsetof({c}, {f}));' for f, _ in py._fields_]
    src, exe = tmp_path / "layout.c", tmp_path / "layout"
    src.write_text("\n".join(lines + ["return 0; }"]))
    subprocess.check_call(["gcc", "-std=c11", "-o", str(exe), str(src)])
    got = [int(x) for x in subprocess.check_output([str(exe)]).split()]
    want = [M.MIMO_DTYPE_INT4, M.MIMO_INT4_K_SLOT_BYTES, M.MIMO_INT4_V_SLOT_BYTES, M.MIMO_SELECT_MAX_SLOTS]
    for py in structs.values():
        want += [C.sizeof(py)] + [getattr(py, f).offset for f, _ in py._fields_]
    assert got == want


@gpu
@pytest.mark.parametrize("fmt", [BF16, E4M3, INT4])
@pytest.mark.parametrize("q_len", [1, 3])
def test_weights_of_a_query_row_without_a_number(fmt, q_len):
    """A query row of NaN or infinities, whose log-sum-exp is no number: it adds nothing, the other rows
    what they add without it, bit for bit."""
    g, r = gen(26), np.random.default_rng(26)
    lens = [900, 131]
    table, pages = R.table_of(lens, r)
    k, v, kd, vd = R.random_cache(fmt, pages, g)
    q = torch.randn((2 * q_len, 64, 192), generator=g, device="cuda").bfloat16()
    kw = dict(max_seq_len=900, num_kv_heads=4, rope_base=1e7, k_cache=k, block_table=table, num_pages=pages, cache_dtype=fmt,
              k_dequant=kd, q_len=q_len)
    _, lse = M.mimo_attn_decode(q, R.i32(lens), window=0, cache_kind=PAGED, v_cache=v, v_dequant=vd, **kw)
    before = torch.rand((2, 4, 900), generator=g, device="cuda")
    M.status_poll()

    def run(q, lse):
        return M.mimo_attn_weights(q, lse, before.clone(), R.i32(lens), **kw)
    for bad in (float("nan"), float("inf"), -float("inf")):
        for what in (slice(None), slice(0, 1), slice(100, 101)):
            q2, l2 = q.clone(), lse.clone()
            q2[0, 5, what] = bad          # head 5: KV head 0
            q2[q_len, 40, what] = bad     # head 40: KV head 2
            l2[0, 5], l2[q_len, 40] = float("nan"), float("inf")
            got, want = run(q2, l2), run(q, l2)
            assert torch.isfinite(got).all() and torch.equal(got, want)
    assert M.status_poll() in (0, M.MIMO_STATUS_RANGE)


def _from_two_threads(fn, calls, times):
    """Return codes of a C entry point called over and over from a host thread per argument struct, each
    on a stream of its own."""
    import threading
    codes = [set() for _ in calls]
    streams = [torch.cuda.Stream() for _ in calls]
    start = threading.Barrier(len(calls))

    def work(args, stream, seen):
        ref, handle = C.byref(args), stream.cuda_stream
        start.wait()
        for _ in range(times):
            seen.add(fn(ref, handle))
    threads = [threading.Thread(target=work, args=x) for x in zip(calls, streams, codes)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    return codes


@gpu
def test_select_from_two_host_threads():
    """Rows whose kernels take different amounts of shared memory, selected at the same time."""
    calls, sets = [], []
    for n in (390000, 150000):
        scores = torch.rand((1, 4, n), generator=gen(n), device="cuda")
        idx, counts, lens = (torch.zeros(s, dtype=torch.int32, device="cuda") for s in ((1, 4, 500), (1,), (1,)))
        lens.fill_(n)
        a = M.MimoSelectArgs()
        a.num_seqs, a.num_kv_heads, a.score_stride, a.max_seq_len, a.keep = 1, 4, n, n, 500
        a.scores, a.seq_lens, a.idx, a.counts = (t.data_ptr() for t in (scores, lens, idx, counts))
        calls.append(a)
        sets.append((scores, lens, idx, counts, select_ref(scores, [n], 500, 0, 0)))
    torch.cuda.synchronize()
    assert _from_two_threads(M.lib().mimo_kv_select, calls, 20000) == [{M.MIMO_OK}] * 2
    for _, _, idx, _, want in sets:
        assert torch.equal(idx.cpu(), want)
    assert M.status_poll() == 0


@gpu
@pytest.mark.parametrize("fmt", [BF16, E4M3])
def test_weights_from_two_host_threads(fmt):
    """One token and eight drafts: other amounts of shared memory of the same kernel."""
    g = gen(27)
    k, _, kd, _ = R.random_cache(fmt, 2, g)
    table, lens, calls, sets = R.i32([[0, 1]]), R.i32([200]), [], []
    for q_len in (1, 8):
        q = torch.randn((q_len, 64, 192), generator=g, device="cuda").bfloat16()
        lse, scores = torch.full((q_len, 64), 5.0, device="cuda"), torch.zeros((1, 4, 256), device="cuda")
        a = M.MimoWeightsArgs()
        a.layer = M.make_layer(4, 1e7, 0)
        a.batch, a.q_len, a.max_seq_len, a.score_stride, a.max_pages, a.num_pages, a.cache_dtype = 1, q_len, 200, 256, 2, 2, fmt
        a.q, a.lse, a.seq_lens, a.k_cache, a.block_table, a.scores = (t.data_ptr() for t in (q, lse, lens, k, table, scores))
        a.k_dequant = kd.data_ptr() if fmt == E4M3 else None
        calls.append(a)
        sets.append((q, lse, scores))
    torch.cuda.synchronize()
    assert _from_two_threads(M.lib().mimo_attn_weights, calls, 20000) == [{M.MIMO_OK}] * 2
    assert M.status_poll() == 0


@gpu
def test_weights_ignore_what_lies_behind_e4m3():
    def spoil(k, table):
        k[int(table[0, 1]), 40:] = 0x7F  # NaN
    check_weights([168], E4M3, seed=23, edit=spoil)


def test_tensors_of_another_device_are_refused_on_any_stream(monkeypatch):
    other = type("T", (), dict(is_cuda=True, device=torch.device("cuda", 1)))()
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)
    for stream in (None, 0, 12345678, type("S", (), dict(cuda_stream=4096))()):
        with pytest.raises(ValueError, match="current device"):
            M._stream(stream, other)
    here = type("T", (), dict(is_cuda=True, device=torch.device("cuda", 0)))()
    assert M._stream(12345678, here) == 12345678


def test_python_refusals_of_index_tensors():
    """The small tensors of the eviction calls and what decode and append take for evicted caches: a
    64-bit, short or strided one is refused, not read as something else."""
    i = lambda *shape: torch.zeros(shape, dtype=torch.int32)
    s, n, q = torch.zeros((2, 4, 64)), torch.ones(2, dtype=torch.int32), torch.zeros((4, 64, 192), dtype=torch.bfloat16)
    wide = torch.zeros(4, dtype=torch.int32)[::2]
    bad32 = (n.long(), n[:1], wide, n.float())
    wkw = dict(max_seq_len=32, num_kv_heads=4, rope_base=1e7, k_cache=s, block_table=i(2, 1), num_pages=1, q_len=2, stream=0)
    for bad in bad32:
        with pytest.raises(ValueError, match="seq_lens"):
            M.mimo_kv_select(s, bad, max_seq_len=32, keep=8, stream=0)
        with pytest.raises(ValueError, match="seq_lens"):
            M.mimo_attn_weights(q, torch.zeros((4, 64)), s, bad, **wkw)
        with pytest.raises(ValueError, match="positions"):
            M.mimo_attn_weights(q, torch.zeros((4, 64)), s, n, positions=bad, **wkw)
        with pytest.raises(ValueError, match="positions"):
            M.mimo_attn_decode(q, n, max_seq_len=32, num_kv_heads=4, rope_base=1e7, window=0, cache_kind=PAGED, k_cache=s,
                               v_cache=s, block_table=i(2, 1), num_pages=1, q_len=2, positions=bad, stream=0)
        with pytest.raises(ValueError, match="slots"):
            M.mimo_kv_append(torch.zeros((2, 4, 192)).bfloat16(), torch.zeros((2, 4, 128)).bfloat16(), n, n, rope_base=1e7,
                             cache_kind=PAGED, k_cache=s, v_cache=s, num_seqs=2, block_table=i(2, 1), num_pages=1, slots=bad,
                             stream=0)
    for bad in (n.long(), wide, n.float()):
        with pytest.raises(ValueError, match="counts"):
            M.mimo_kv_gather(s, s, i(2, 1), s, s, i(2, 1), bad, num_kv_heads=4, num_pages=1, num_pages_out=1, stream=0)
    for bad in (torch.zeros((2, 64)), torch.zeros((4, 64)).double(), torch.zeros((4, 128))[:, ::2], i(4, 64)):
        with pytest.raises(ValueError, match="lse"):
            M.mimo_attn_weights(q, bad, s, n, **wkw)
    for bad in (i(2, 1).long(), i(1, 1), i(2, 4)[:, ::2], i(2)):
        with pytest.raises(ValueError, match="block_table"):
            M.mimo_attn_weights(q, torch.zeros((4, 64)), s, n, **{**wkw, "block_table": bad})
    for bad in (i(2, 1).long(), i(2, 4)[:, ::2]):
        for tables in ((bad, i(2, 1)), (i(2, 1), bad)):
            with pytest.raises(ValueError, match="block_table"):
                M.mimo_kv_gather(s, s, tables[0], s, s, tables[1], n, num_kv_heads=4, num_pages=1, num_pages_out=1, stream=0)


@gpu
def test_gather_reports_a_negative_count():
    g = gen(10)
    k, v, _, _ = R.random_cache(BF16, 3, g)
    ko, vo = _empty(BF16, 2, 4)
    M.mimo_kv_gather(k, v, R.i32([[0], [1]]), ko, vo, R.i32([[0], [1]]), R.i32([-1, 2]), num_kv_heads=4, num_pages=3,
                     num_pages_out=2)
    assert M.status_poll() == M.MIMO_STATUS_BAD_INDEX
    assert not ko[0].any() and torch.equal(ko[1, :2], k[1, :2]) and not ko[1, 2:].any()


@gpu
@pytest.mark.parametrize("fmt", [BF16, E4M3, INT4])
@pytest.mark.parametrize("q_len", [2, 4, 8])
def test_decode_drafts_with_positions(fmt, q_len):
    """Draft tokens over an evicted cache: slots and rotary positions differ, in every cache format."""
    g, r = gen(28), np.random.default_rng(28)
    lens, pos = [200, 3000, 9], [5000, 120000, 8]
    table, pages = R.table_of(lens, r)
    k, v, kd, vd = R.random_cache(fmt, pages, g)
    q = torch.randn((3 * q_len, 64, 192), generator=g, device="cuda").bfloat16()
    out, lse = M.mimo_attn_decode(q, R.i32(lens), max_seq_len=3000, num_kv_heads=4, rope_base=1e7, window=0, cache_kind=PAGED,
                                  k_cache=k, v_cache=v, block_table=table, num_pages=pages, cache_dtype=fmt, k_dequant=kd,
                                  v_dequant=vd, q_len=q_len, positions=R.i32(pos))
    assert M.status_poll() == 0
    kv, vv = R.slots_of(k, fmt, 192, kd), R.slots_of(v, fmt, 128, vd)
    for s, n in enumerate(lens):
        me, sl = torch.arange(n - q_len, n, device="cuda"), slice(s * q_len, (s + 1) * q_len)
        R.Row(q[sl], R.pages_of(kv, table[s], n), R.pages_of(vv, table[s], n), torch.arange(n, device="cuda"), me, 1e7,
              pos=me - (n - 1) + pos[s], p_step=2.0 ** -8 if fmt == BF16 else 2.0 ** -10).check(out[sl], lse[sl], f"sequence {s}")


@gpu
@pytest.mark.parametrize("fmt", [BF16, INT4])
def test_eviction_step_captured(fmt):
    """Append, decode, weights, selection and gather in one graph, replayed on other contents: bit for bit
    what the calls give one by one."""
    g, r = gen(29), np.random.default_rng(29)
    lens, keep = [1500, 130, 900], 200
    table, pages = R.table_of(lens, r)
    table2, pages2 = R.table_of([keep] * 3, r)
    k, v, _, _ = R.random_cache(fmt, pages, g)
    fresh = _empty(fmt, pages2, 4)
    state = dict(k=k, v=v, k2=fresh[0], v2=fresh[1], scores=torch.zeros((3, 4, 1500), device="cuda"),
                 q=torch.zeros((3, 64, 192), device="cuda").bfloat16(), kn=torch.zeros((3, 4, 192), device="cuda").bfloat16(),
                 vn=torch.zeros((3, 4, 128), device="cuda").bfloat16(), lens=R.i32([1, 1, 1]), pos=R.i32([0, 0, 0]))
    seq = R.i32([0, 1, 2])

    def step(t):
        paged = dict(k_cache=t["k"], block_table=table, num_pages=pages, cache_dtype=fmt, rope_base=1e7)
        M.mimo_kv_append(t["kn"], t["vn"], t["pos"], seq, cache_kind=PAGED, v_cache=t["v"], num_seqs=3, **paged)
        kw = dict(max_seq_len=1500, num_kv_heads=4, **paged)
        out, lse = M.mimo_attn_decode(t["q"], t["lens"], window=0, cache_kind=PAGED, v_cache=t["v"], **kw)
        M.mimo_attn_weights(t["q"], lse, t["scores"], t["lens"], **kw)
        idx, counts, kept = M.mimo_kv_select(t["scores"], t["lens"], max_seq_len=1500, keep=keep, recent=16, first=4)
        M.mimo_kv_gather(t["k"], t["v"], table, t["k2"], t["v2"], table2, counts, num_kv_heads=4, num_pages=pages,
                         num_pages_out=pages2, idx=idx, cache_dtype=fmt)
        return out, lse, idx, counts, kept
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = step(state)
    graph.replay()
    for seed in (1, 2):
        new = {n: torch.randn(state[n].shape, generator=gen(seed), device="cuda").bfloat16() for n in ("q", "kn", "vn")}
        new.update(lens=R.i32(lens), pos=R.i32([n - 1 for n in lens]))
        for n, t in new.items():
            state[n].copy_(t)
        alone = {n: t.clone() for n, t in state.items()}
        graph.replay()
        want = step(alone)
        for a, b in zip(got, want):
            assert torch.equal(a, b)
        for n in ("k", "v", "k2", "v2", "scores"):
            assert torch.equal(state[n].view(torch.uint8), alone[n].view(torch.uint8))
    assert M.status_poll() == 0


@gpu
@pytest.mark.parametrize("q_len", [1, 4])
@pytest.mark.parametrize("lens", [[0, 4000, 0, 0, 77, 0], [300, 0, 0, 450, 0, 9]])
def test_padded_batch_over_4_bits(lens, q_len):
    """Rows of a batch that hold no sequence (length 0) are reported; the others are served."""
    g, r = gen(31), np.random.default_rng(31)
    table, pages = R.table_of(lens, r)
    k, v, _, _ = R.random_cache(INT4, pages, g)
    q = torch.randn((len(lens) * q_len, 64, 192), generator=g, device="cuda").bfloat16()
    kw = dict(max_seq_len=max(lens), num_kv_heads=4, rope_base=1e7, k_cache=k, block_table=table, num_pages=pages,
              cache_dtype=INT4, q_len=q_len)
    out, lse = M.mimo_attn_decode(q, R.i32(lens), window=0, cache_kind=PAGED, v_cache=v, **kw)
    assert M.status_poll() == M.MIMO_STATUS_BAD_INDEX
    scores = torch.zeros((len(lens), 4, max(lens)), device="cuda")
    M.mimo_attn_weights(q, lse, scores, R.i32(lens), **kw)
    assert M.status_poll() == M.MIMO_STATUS_BAD_INDEX
    kv, vv = R.slots_of(k, INT4, 192), R.slots_of(v, INT4, 128)
    for s, n in enumerate(lens):
        if n == 0:
            assert not scores[s].any()
            continue
        sl = slice(s * q_len, (s + 1) * q_len)
        R.Row(q[sl], R.pages_of(kv, table[s], n), R.pages_of(vv, table[s], n), torch.arange(n, device="cuda"),
              torch.arange(n - q_len, n, device="cuda"), 1e7).check(out[sl], lse[sl], f"sequence {s}")
        # (as for a decode's own log-sum-exp: a KV head's 16 heads, for every draft)
        assert float((scores[s].double().sum(-1) - 16 * q_len).abs().max()) < 16 * q_len * 2e-3
    check_select(scores, lens, 100, 5)


@gpu
@pytest.mark.parametrize("fmt", [BF16, E4M3, INT4])
def test_pages_beyond_four_gigabytes(fmt):
    """The calls on the last pages of a large pool: bit for bit what they give on a small one."""
    g, r = gen(32), np.random.default_rng(32)
    lens = [700, 3, 129]
    table, pages = R.table_of([n + 1 for n in lens], r)
    k, v, kd, vd = R.random_cache(fmt, pages, g)
    q = torch.randn((3, 64, 192), generator=g, device="cuda").bfloat16()
    kn, vn = (torch.randn((3, 4, d), generator=g, device="cuda").bfloat16() for d in (192, 128))
    table2, pages2 = R.table_of([100] * 3, r)
    big = -(-(1 << 32) // (v[0].numel() * v.element_size())) + 50

    def run(k, v, at, k2, v2, at2, n, n2):
        t1, t2 = torch.where(table >= 0, table + at, table), table2 + at2
        fm = dict(cache_dtype=fmt, k_dequant=kd)
        M.mimo_kv_append(kn, vn, R.i32(lens), R.i32([0, 1, 2]), rope_base=1e7, cache_kind=PAGED, k_cache=k, v_cache=v,
                         num_seqs=3, block_table=t1, num_pages=n, v_dequant=vd, **fm)
        now = R.i32([x + 1 for x in lens])
        kw = dict(max_seq_len=701, num_kv_heads=4, rope_base=1e7, k_cache=k, block_table=t1, num_pages=n, **fm)
        out, lse = M.mimo_attn_decode(q, now, window=0, cache_kind=PAGED, v_cache=v, v_dequant=vd, **kw)
        scores = torch.zeros((3, 4, 704), device="cuda")
        M.mimo_attn_weights(q, lse, scores, now, **kw)
        idx, counts, _ = M.mimo_kv_select(scores, now, max_seq_len=701, keep=100)
        M.mimo_kv_gather(k, v, t1, k2, v2, t2, counts, num_kv_heads=4, num_pages=n, num_pages_out=n2, idx=idx, cache_dtype=fmt)
        return out, lse, scores, idx
    small, small2 = (k.clone(), v.clone()), _empty(fmt, pages2, 4)
    want = run(*small, 0, *small2, 0, pages, pages2)
    pool, pool2 = _empty(fmt, big, 4), _empty(fmt, big, 4)
    for a, b in zip(pool, (k, v)):
        a[big - pages:] = b
    got = run(*pool, big - pages, *pool2, big - pages2, big, big)
    assert M.status_poll() == 0
    for a, b in zip(got, want):
        assert torch.equal(a, b)
    for a, b, n in zip(pool + pool2, small + small2, (pages, pages, pages2, pages2)):
        assert torch.equal(a[big - n:].view(torch.uint8), b.view(torch.uint8))
        assert not a[:big - n].view(torch.uint8).any()
    del pool, pool2
    torch.cuda.empty_cache()
