"""Paged key/value cache on the GPU: append, attention and gather against the plain fp64 forms of
tests/_paged.py, at the lengths, masks, layouts and values where they can go wrong, and a serving run of
them together against the dense forward."""
import math

import numpy as np
import pytest
import torch

import column_sparse_masked_b200 as fm
from column_sparse_masked_b200 import workloads as wl

import _paged as ref
from _paged import Cache, HALF_BF16, bf16, f64

pytestmark = pytest.mark.gpu


def i32(x):
    return torch.tensor(np.asarray(x), dtype=torch.int32).cuda()


@pytest.fixture(autouse=True)
def clean_status():
    fm.get_status()
    yield
    assert fm.get_status() == 0


# ---------------------------------------------------------------------------
# attention
# ---------------------------------------------------------------------------
def masks(kind, B, Hm, n, seed, rows):
    rng = np.random.default_rng(seed)
    v = np.zeros((4, B, Hm, n), np.int32)
    for b in range(B):
        for h in range(Hm):
            if kind == "random":
                v[:, b, h] = wl.random_interval_vectors(rng, n + 2, n)
            elif kind == "doc":
                v[:, b, h] = wl.causal_document_vectors(wl.doc_lengths_uniform(rng, n, 20, 150))
                v[0, b, h][v[0, b, h] == n] = n + rows
            elif kind == "window":
                v[:, b, h] = wl.prefix_window_vectors(n, 16, 90)
            elif kind == "tiles":  # whole blocks of keys dropped, none visible in the last block of some
                v[:, b, h] = wl.drop_key_tiles(wl.causal_vectors(n), rng, 0.6, 32)
                v[1, b, h] = n + rows
            elif kind == "nothing":
                v[0, b, h], v[1, b, h] = -2 ** 31, 2 ** 31 - 1
            elif kind == "nothing_pair":  # the two intervals cover every row together
                v[:, b, h] = np.array([-5, n // 2, n // 2, n + rows + 1])[:, None]
    return [torch.from_numpy(x).cuda() for x in v]


def check_attention(q, cache, lens, vec=(None,) * 4, **kw):
    o, lse = fm.paged_attention(q, cache.k, cache.v, cache.table, i32(lens), *vec, **cache.kw, **kw)
    st = kw.get("start")
    ro, rl, to, tl = ref.attention(q, cache, lens, vec, None if st is None else st.cpu().tolist(),
                                   kw.get("causal", True), kw.get("scale"))
    eo, el = f64(o), f64(lse)
    empty = np.isneginf(rl)
    assert np.array_equal(np.isneginf(el), empty)
    assert not np.isnan(eo).any() and not np.isnan(el).any()
    worst = (np.abs(eo - ro) / np.maximum(to, 1e-30)).max() if eo.size else 0
    assert (np.abs(eo - ro) <= to).all(), f"O off by {worst:.2f} of its bound"
    assert (np.abs(el[~empty] - rl[~empty]) <= tl[~empty]).all(), "LSE"
    assert (eo[np.swapaxes(empty, 1, 2)] == 0).all()
    return o, lse


def case_q(B, Nq, Hq, d, seed=1):
    g = torch.Generator().manual_seed(seed)
    return torch.randn(B, Nq, Hq, d, generator=g).bfloat16().cuda()


@pytest.mark.parametrize("bits", [16, 4])
@pytest.mark.parametrize("lens,Nq,Hq,Hkv,d,page", [
    ([1], 1, 1, 1, 64, 16),
    ([0, 1, 2, 15, 16, 17], 1, 2, 2, 128, 16),
    ([31, 32, 33, 63, 64, 65, 127, 128, 129], 1, 4, 2, 64, 32),
    ([257, 0, 640], 1, 8, 1, 128, 64),
    ([1003], 1, 3, 3, 128, 256),
    ([777, 40], 2, 12, 4, 64, 128),
    ([300, 5, 161], 5, 6, 2, 128, 16),
    ([200, 8], 8, 8, 2, 64, 64),
    ([411, 3], 16, 8, 1, 128, 32),
    ([90], 33, 5, 1, 64, 16),
    ([2500], 1, 16, 2, 128, 128),
])
def test_attention_lengths(bits, lens, Nq, Hq, Hkv, d, page):
    check_attention(case_q(len(lens), Nq, Hq, d), Cache(7, lens, Hkv, d, page, bits).cuda(), lens)


@pytest.mark.parametrize("bits", [16, 4])
@pytest.mark.parametrize("kind", ["random", "doc", "window", "tiles", "nothing", "nothing_pair"])
@pytest.mark.parametrize("Hm", [1, 4])
@pytest.mark.parametrize("Nq", [1, 3])
def test_attention_masks(bits, kind, Hm, Nq):
    lens = [430, 77, 1, 256]
    cache = Cache(11, lens, 2, 128, 32, bits).cuda()
    check_attention(case_q(4, Nq, 4, 128), cache, lens, masks(kind, 4, Hm, max(lens), 3, Nq))


@pytest.mark.parametrize("bits", [16, 4])
def test_attention_mask_pairs_and_short_vectors(bits):
    """One pair alone, and vectors shorter than the cache: later keys have no interval."""
    lens = [300, 150]
    cache, q = Cache(12, lens, 2, 64, 16, bits).cuda(), case_q(2, 2, 4, 64)
    m = [x[..., :101].contiguous() for x in masks("random", 2, 1, 300, 4, 2)]
    check_attention(q, cache, lens, [m[0], m[1], None, None])
    check_attention(q, cache, lens, [None, None, m[2], m[3]])
    empty = [x[..., :0].contiguous() for x in m]
    check_attention(q, cache, lens, empty)


@pytest.mark.parametrize("bits", [16, 4])
def test_attention_start_causal_scale(bits):
    lens = [260, 90, 17]
    cache, q = Cache(13, lens, 2, 64, 32, bits).cuda(), case_q(3, 4, 4, 64)
    check_attention(q, cache, lens, start=i32([100, 0, 500]))
    check_attention(q, cache, lens, start=i32([-3, -9, 2]))     # rows in front of the first key see nothing
    check_attention(q, cache, lens, causal=False)
    check_attention(q, cache, lens, scale=0.03)
    check_attention(q, cache, lens, masks("random", 3, 4, 260, 5, 4), causal=False, start=i32([50, 3, 8]))


@pytest.mark.parametrize("bits", [16, 4])
@pytest.mark.parametrize("what", [float("nan"), float("inf"), -float("inf")])
def test_attention_unseen_keys_have_no_influence(bits, what):
    """NaN and infinities behind the last key, in hidden keys (one head's or everyone's) and in pages of
    nobody; every row sees finite keys only."""
    lens, Hq = [200, 45, 96], 4
    cache = Cache(14, lens, 2, 128, 32, bits)
    vec = masks("random", 3, Hq, 200, 6, 3)
    hidden_all = np.arange(200) % 7 == 3
    for x, val in zip(vec, (-1, 10 ** 6, 0, 0)):
        x[:, :, torch.from_numpy(hidden_all).cuda()] = val
    # a key that only head 1 of KV head 0 does not see, next to rows that do: NaN would be right for those,
    # so only keys hidden from every head of a KV head are poisoned, but for each KV head its own
    lo, hi, lo2, hi2 = (f64(x).astype(np.int64) for x in vec)
    for b, n in enumerate(lens):
        for kv in range(2):
            rows = [(h, n - 3 + i) for h in (2 * kv, 2 * kv + 1) for i in range(3)]
            seen = np.zeros(n, bool)
            for h, p in rows:
                seen |= ref.visible(p, n, True, (lo, hi, lo2, hi2), b, h)
            room = -(-n // cache.page) * cache.page
            for j in list(np.nonzero(~seen)[0]) + list(range(n, room)):
                page, slot = int(cache.table[b, j // cache.page]), j % cache.page
                for t in ((cache.k, cache.v) if bits == 16 else (cache.ks, cache.vs)):
                    t[page, kv, slot] = what
    clean = Cache(14, lens, 2, 128, 32, bits)
    cache, clean, q = cache.cuda(), clean.cuda(), case_q(3, 3, Hq, 128)
    o, lse = fm.paged_attention(q, cache.k, cache.v, cache.table, i32(lens), *vec, **cache.kw)
    check_attention(q, clean, lens, vec)
    ro, rl = fm.paged_attention(q, clean.k, clean.v, clean.table, i32(lens), *vec, **clean.kw)
    assert torch.equal(o, ro) and torch.equal(lse, rl)


@pytest.mark.parametrize("Nq", [1, 3])
def test_attention_nan_reaches_only_rows_that_see_it(Nq):
    """A key of NaN that one head sees and another (same KV head) does not."""
    n, Hq = 150, 4
    cache, q = Cache(15, [n], 2, 64, 16, 16), case_q(1, Nq, Hq, 64)
    vec = [torch.zeros(1, Hq, n, dtype=torch.int32, device="cuda") for _ in range(4)]
    for j in (5, 70, 149):
        vec[0][0, 1, j], vec[1][0, 1, j] = -1, 10 ** 6  # hidden from head 1
        cache.v[int(cache.table[0, j // 16]), 0, j % 16] = float("nan")
    clean = Cache(15, [n], 2, 64, 16, 16).cuda()
    cache = cache.cuda()
    o, _ = fm.paged_attention(q, cache.k, cache.v, cache.table, i32([n]), *vec)
    ro, _ = fm.paged_attention(q, clean.k, clean.v, clean.table, i32([n]), *vec)
    assert torch.isnan(o[:, -1, 0]).all()
    assert torch.equal(o[:, :, 1:], ro[:, :, 1:])


@pytest.mark.parametrize("bits", [16, 4])
@pytest.mark.parametrize("lens,width,B", [([150], None, 1), ([60] * 90, None, 90), ([3000, 40], 60, 2)])
def test_attention_nan_scores_are_not_taken_for_hidden_ones(bits, lens, width, B):
    """A row of q with a NaN, and a key of NaN that every row of one KV head sees, give NaN in O and LSE of those rows
    and leave the others alone: one item per CTA, per warp, and cut."""
    cache, q = Cache(29, lens, 2, 64, 64, bits, width=width), case_q(B, 2, 4, 64)
    clean = Cache(29, lens, 2, 64, 64, bits, width=width).cuda()
    want, wl_ = fm.paged_attention(q, clean.k, clean.v, clean.table, i32(lens), **clean.kw)
    bad_q = q.clone()
    bad_q[0, 1, 2, 5] = float("nan")
    o, lse = fm.paged_attention(bad_q, clean.k, clean.v, clean.table, i32(lens), **clean.kw)
    assert torch.isnan(o[0, 1, 2]).all() and torch.isnan(lse[0, 2, 1])
    o[0, 1, 2], lse[0, 2, 1] = want[0, 1, 2], wl_[0, 2, 1]
    assert torch.equal(o, want) and torch.equal(lse, wl_)
    (cache.k if bits == 16 else cache.ks)[int(cache.table[0, 0]), 1, 3] = float("nan")
    cache = cache.cuda()
    o, lse = fm.paged_attention(q, cache.k, cache.v, cache.table, i32(lens), **cache.kw)
    assert torch.isnan(o[0, :, 2:]).all() and torch.isnan(lse[0, 2:]).all()
    assert torch.equal(o[0, :, :2], want[0, :, :2]) and torch.equal(o[1:], want[1:]) and torch.equal(lse[1:], wl_[1:])


@pytest.mark.parametrize("bits", [16, 4])
def test_cache_of_more_than_32_bits(bits):
    """Pages whose offsets pass 2^32 bytes and, for bf16, 2^31 values: the last pages of the cache and the first ones
    give what the same pages give in a small cache."""
    Hkv, page, d, lens = 2, 256, 128, [700, 300]
    small = Cache(30, lens, Hkv, d, page, bits, spare=0).cuda()
    P = (2 ** 24 if bits == 16 else 2 ** 26) // (Hkv * page) + 8
    big = [None if x is None else torch.empty((P,) + x.shape[1:], dtype=x.dtype, device="cuda")
           for x in (small.k, small.v, small.ks, small.vs)]
    assert big[0].numel() * big[0].element_size() > 2 ** 32
    n = small.k.shape[0]
    where = torch.tensor([P - 1, 0, P - 2, P - 5, 1, P - 3][:n], device="cuda")
    for x, y in zip(big, (small.k, small.v, small.ks, small.vs)):
        if x is not None:
            x[where] = y
    table = torch.where(small.table < 0, -1, where[small.table.clamp(min=0).long()]).int()
    kw = {} if bits == 16 else {"k_scales": big[2], "v_scales": big[3]}
    q, lens_ = case_q(2, 3, 8, d), i32(lens)
    for a, b in zip(fm.paged_attention(q, big[0], big[1], table, lens_, **kw),
                    fm.paged_attention(q, small.k, small.v, small.table, lens_, **small.kw)):
        assert torch.equal(a, b)
    for a, b in zip(fm.paged_gather(big[0], big[1], table, lens_, 700, **kw),
                    fm.paged_gather(small.k, small.v, small.table, lens_, 700, **small.kw)):
        assert torch.equal(a, b)
    k = case_q(2, 5, Hkv, d, 3)
    fm.paged_append(k, k, big[0], big[1], table, i32([250, 290]), **kw)
    fm.paged_append(k, k, small.k, small.v, small.table, i32([250, 290]), **small.kw)
    for x, y in zip(big, (small.k, small.v, small.ks, small.vs)):
        if x is not None:
            assert torch.equal(x[where], y)


def test_attention_infinite_value_in_a_seen_key():
    n = 100
    cache, q = Cache(16, [n], 1, 64, 16, 16), case_q(1, 1, 2, 64)
    vec = [torch.zeros(1, 2, n, dtype=torch.int32, device="cuda") for _ in range(4)]
    vec[0][0, 1, 40], vec[1][0, 1, 40] = 0, 1000
    cache.v[int(cache.table[0, 40 // 16]), 0, 40 % 16, 9] = float("inf")
    cache = cache.cuda()
    o, _ = fm.paged_attention(q, cache.k, cache.v, cache.table, i32([n]), *vec)
    assert o[0, 0, 0, 9] == float("inf") and torch.isfinite(o[0, 0, 0, :9]).all() and torch.isfinite(o[0, 0, 1]).all()


@pytest.mark.parametrize("bits", [16, 4])
def test_attention_layouts(bits):
    """Rows out of a fused projection, a broadcast row, a table that is a slice of a wider one, caller's outputs
    and workspace."""
    lens = [130, 61]
    cache = Cache(17, lens, 2, 128, 64, bits).cuda()
    fused = case_q(2, 3, 8, 128)
    check_attention(fused[:, :, 2:6], cache, lens)
    check_attention(fused[:, :1, :4].expand(2, 3, 4, 128), cache, lens)
    wide = torch.full((4, 40), -7, dtype=torch.int32, device="cuda")
    wide[::2, 3:3 + cache.table.shape[1]] = cache.table
    q = fused[:, :, :4]
    o, lse = check_attention(q, cache, lens)
    w = wide[::2, 3:3 + cache.table.shape[1]]
    out = (torch.full_like(o, 9.0), torch.full_like(lse, 9.0))
    ws = torch.full((1 << 26,), 255, dtype=torch.uint8, device="cuda")
    o2, l2 = fm.paged_attention(q, cache.k, cache.v, w, i32(lens), out=out, workspace=ws, **cache.kw)
    assert o2 is out[0] and torch.equal(o, o2) and torch.equal(lse, l2)
    with pytest.raises(fm.FlashMaskError, match="workspace"):
        fm.paged_attention(q, cache.k, cache.v, w, i32(lens), workspace=ws[:0], **cache.kw)


@pytest.mark.parametrize("bits", [16, 4])
def test_attention_many_sequences(bits):
    """More sequences than CTAs, most of them short or empty, sharing a prefix page."""
    rng = np.random.default_rng(3)
    lens = [int(x) for x in rng.integers(0, 90, 400)]
    lens[7], lens[399] = 700, 0
    cache = Cache(18, lens, 1, 64, 16, bits)
    for b in range(400):
        if lens[b] > 16:
            cache.table[b, 0] = cache.table[7, 0]
    check_attention(case_q(400, 1, 2, 64), cache.cuda(), lens)


@pytest.mark.parametrize("bits", [16, 4])
@pytest.mark.parametrize("Hm,cap", [(0, 0), (1, 0), (4, 3)])
def test_attention_many_short_sequences(bits, Hm, cap):
    """More items than a device takes at once, each of a few tiles: whole items per warp."""
    rng = np.random.default_rng(4)
    lens = [int(x) for x in rng.integers(0, 250, 150)]
    lens[3], lens[149] = 256, 0
    cache = Cache(25, lens, 2, 128, 32, bits).cuda()
    vec = (None,) * 4 if Hm == 0 else masks("random", 150, Hm, 256, 5, 2)
    fm.set_max_ctas(cap)
    try:
        check_attention(case_q(150, 2, 4, 128), cache, lens, vec)
    finally:
        fm.set_max_ctas(0)


@pytest.mark.parametrize("bits", [16, 4])
@pytest.mark.parametrize("Hm", [0, 1, 8])
@pytest.mark.parametrize("shape", ["short", "two_waves", "many", "long", "wide_table"])
def test_attention_more_rows_than_a_block(bits, Hm, shape):
    """40 rows of a KV head: several blocks of rows, of 8, 16 and (bf16 with room for long sequences) 32, one
    item per CTA, per warp, and cut."""
    d, Nq, width = 128, 10, None
    lens = {"short": [61, 200], "two_waves": [600] + [9] * 59, "many": [120, 3] * 20, "long": [5100, 40],
            "wide_table": [700, 90]}[shape]
    if shape == "wide_table":
        width = 1800
    if shape in ("two_waves", "many"):
        Nq, d = 5, 64 if shape == "many" else 128
    cache = Cache(26, lens, 2, d, 64, bits, width=width).cuda()
    vec = (None,) * 4 if Hm == 0 else masks("random", len(lens), Hm, max(lens), 15, Nq)
    check_attention(case_q(len(lens), Nq, 8, d), cache, lens, vec)


@pytest.mark.parametrize("bits", [16, 4])
@pytest.mark.parametrize("G", [3, 5, 12, 40])
@pytest.mark.parametrize("lens,width", [([150, 33], None), ([60, 64] * 40, None), ([700, 90], 60)])
def test_attention_mask_heads_that_do_not_divide_a_block(bits, G, lens, width):
    """A mask head for each q-head, with groups of heads that end inside a block of rows: one item per CTA, per warp,
    and cut."""
    Nq = 7 if len(lens) == 2 else 2
    cache = Cache(31, lens, 2, 64, 64, bits, width=width).cuda()
    vec = masks("random", len(lens), 2 * G, max(lens), 16, Nq)
    check_attention(case_q(len(lens), Nq, 2 * G, 64), cache, lens, vec)


@pytest.mark.parametrize("bits", [16, 4])
@pytest.mark.parametrize("Hm,width", [(0, None), (1, None), (2, None), (0, 48), (1, 48), (2, 48)])
def test_attention_more_sequences_than_shared_memory_holds(bits, Hm, width):
    rng = np.random.default_rng(6)
    lens = [int(x) for x in rng.integers(0, 70, 700)]
    lens[0] = lens[511] = lens[699] = 0
    if width:
        lens[5], lens[512], lens[698] = 700, 650, 300
    cache = Cache(27, lens, 2, 64, 16, bits, width=width).cuda()
    vec = (None,) * 4 if Hm == 0 else masks("random", 700, Hm, max(lens), 7, 1)
    check_attention(case_q(700, 1, 2, 64), cache, lens, vec)


@pytest.mark.parametrize("bits", [16, 4])
@pytest.mark.parametrize("width", [None, 80])
def test_attention_positions_at_the_ends_of_their_type(bits, width):
    """start and boundaries anywhere in 32 bits: positions do not wrap."""
    lens, lo, hi = [90, 40, 77, 5], -2 ** 31, 2 ** 31 - 1
    cache, q = Cache(28, lens, 1, 64, 16, bits, width=width).cuda(), case_q(4, 4, 2, 64)
    rng = np.random.default_rng(8)
    for starts in ([hi, hi - 2, lo, lo + 1], [2 ** 30, 2 ** 30 + 5, -2 ** 30, -2 ** 30 - 1], [hi - 1, 3, -1, 0]):
        near = np.array(starts)[None, :, None, None] + rng.integers(-3, 8, (4, 4, 1, 90))
        ends = rng.choice([lo, lo + 1, -1, 0, 1, hi - 1, hi], (4, 4, 1, 90))
        vec = np.clip(np.where(rng.random((4, 4, 1, 90)) < 0.7, near, ends), lo, hi)
        vec = [torch.from_numpy(x.astype(np.int32)).cuda() for x in vec]
        for causal in (False, True):
            check_attention(q, cache, lens, vec, start=i32(starts), causal=causal)
            check_attention(q, cache, lens, start=i32(starts), causal=causal)


@pytest.mark.parametrize("bits", [16, 4])
def test_attention_long(bits):
    """One long sequence split over the whole device; every page also checked through its weights: keys are equal,
    so O is the mean of the values."""
    n, d = 40000, 128
    cache = Cache(19, [n], 2, d, 64, bits).cuda()
    q = torch.zeros(1, 1, 4, d, dtype=torch.bfloat16, device="cuda")
    o, lse = fm.paged_attention(q, cache.k, cache.v, cache.table, i32([n]), **cache.kw)
    v = fm.paged_gather(cache.k, cache.v, cache.table, i32([n]), n, **cache.kw)[1].double()[0]
    mean = v.mean(0).repeat_interleave(2, 0)
    # weights are all 1: only codes times scales, the sums (2^-24 a term, 40000 terms at most) and the
    # result are rounded; the gathered values carry another 2^-8 each
    bound = 2 * HALF_BF16 * v.abs().mean(0).repeat_interleave(2, 0) / math.sqrt(n) * 8 + HALF_BF16 * mean.abs() \
        + n * 2.0 ** -24 * v.abs().mean(0).repeat_interleave(2, 0)
    assert ((o.double()[0, 0] - mean).abs() <= bound).all()
    assert (lse.double() - math.log(n)).abs().max() <= 2.0 ** -20 * (1 + math.log(n))


@pytest.mark.parametrize("bits", [16, 4])
@pytest.mark.parametrize("cap", [1, 2, 5])
@pytest.mark.parametrize("kind,Nq,G,d,page", [
    ("none", 1, 4, 128, 64), ("none", 1, 4, 64, 16), ("none", 4, 4, 128, 32), ("none", 8, 4, 64, 128),
    ("doc", 1, 4, 128, 64), ("random", 2, 4, 64, 32), ("tiles", 3, 4, 128, 16), ("random", 8, 4, 128, 64),
])
def test_attention_few_ctas_walk_many_items(bits, cap, kind, Nq, G, d, page):
    """Runs that hold many items and go round the ring of tiles several times."""
    lens = [900, 0, 33, 4100, 64, 257]
    cache, q = Cache(23, lens, 2, d, page, bits).cuda(), case_q(6, Nq, 2 * G, d)
    vec = (None,) * 4 if kind == "none" else masks(kind, 6, 1, 4100, 8, Nq)
    fm.set_max_ctas(cap)
    try:
        check_attention(q, cache, lens, vec)
    finally:
        fm.set_max_ctas(0)


@pytest.mark.parametrize("bits", [16, 4])
@pytest.mark.parametrize("kind", ["none", "doc"])
def test_attention_calls_in_a_row(bits, kind):
    """Calls queued without waiting between them give the bits of single calls."""
    lens = [1500, 300, 4000]
    cache, q = Cache(24, lens, 2, 128, 64, bits).cuda(), case_q(3, 1, 8, 128)
    vec = (None,) * 4 if kind == "none" else masks(kind, 3, 1, 4000, 8, 1)
    n = i32(lens)
    o, lse = fm.paged_attention(q, cache.k, cache.v, cache.table, n, *vec, **cache.kw)
    torch.cuda.synchronize()
    outs = [fm.paged_attention(q, cache.k, cache.v, cache.table, n, *vec, **cache.kw) for _ in range(40)]
    torch.cuda.synchronize()
    assert all(torch.equal(a, o) and torch.equal(b, lse) for a, b in outs)


@pytest.mark.parametrize("bits", [16, 4])
def test_attention_bad_entries_are_reported_and_left_out(bits):
    lens = [100, 70]
    cache, q = Cache(20, lens, 2, 64, 16, bits).cuda(), case_q(2, 1, 2, 64)
    good = cache.table.clone()
    vec = [torch.zeros(2, 1, 100, dtype=torch.int32, device="cuda") for _ in range(4)]
    vec[0][0, 0, 32:48], vec[1][0, 0, 32:48] = -1, 1000
    o, lse = fm.paged_attention(q, cache.k, cache.v, good, i32(lens), *vec, **cache.kw)
    assert fm.get_status() == 0
    for bad in (-1, cache.k.shape[0], 2 ** 31 - 1, -2 ** 31):
        t = good.clone()
        t[0, 2] = bad
        o2, l2 = fm.paged_attention(q, cache.k, cache.v, t, i32(lens), **cache.kw)
        assert fm.get_status() == -9
        assert torch.equal(o2, o) and torch.equal(l2, lse)  # as if its keys were hidden
    over = fm.paged_attention(q, cache.k, cache.v, good, i32([10 ** 6, 70]), start=i32([99, 69]), **cache.kw)
    assert fm.get_status() == -9
    full = fm.paged_attention(q, cache.k, cache.v, good, i32([100, 70]), start=i32([99, 69]), **cache.kw)
    assert torch.equal(over[0], full[0]) and fm.get_status() == 0


def test_attention_empty_calls():
    cache = Cache(21, [20], 2, 64, 16, 16).cuda()
    o, lse = fm.paged_attention(case_q(1, 0, 4, 64), cache.k, cache.v, cache.table, i32([20]))
    assert o.shape == (1, 0, 4, 64) and lse.shape == (1, 4, 0)
    none = torch.zeros(1, 0, dtype=torch.int32, device="cuda")
    o, lse = fm.paged_attention(case_q(1, 2, 4, 64), cache.k[:0], cache.v[:0], none, i32([0]))
    assert (o == 0).all() and torch.isneginf(lse).all()
    m = torch.zeros(1, 4, 9, dtype=torch.int32, device="cuda")
    o, lse = fm.paged_attention(case_q(1, 2, 4, 64), cache.k, cache.v, none, i32([0]), m, m)
    assert (o == 0).all() and torch.isneginf(lse).all()


# ---------------------------------------------------------------------------
# append
# ---------------------------------------------------------------------------
def tables(n, rot):
    a = np.arange(n)[:, None] * 10000.0 ** (-np.arange(0, rot, 2) / rot)[None]
    return torch.from_numpy(np.cos(a)).float().cuda(), torch.from_numpy(np.sin(a)).float().cuda()


def check_append(bits, B, N, Hq, Hkv, d, page, start, rot, interleaved=False, counts=None, positions=None, seed=31,
                 with_q=True, in_place=False):
    real = [N] * B if counts is None else counts
    cache = Cache(seed, [start[b] + real[b] for b in range(B)], Hkv, d, page, bits).cuda()
    g = torch.Generator().manual_seed(seed + 1)
    qkv = torch.randn(B, N, Hq + 2 * Hkv, d, generator=g).bfloat16().cuda()
    q, k, v = qkv[:, :, :Hq], qkv[:, :, Hq:Hq + Hkv], qkv[:, :, Hq + Hkv:]
    cos, sin = tables(3000, rot) if rot else (None, None)
    before = [f64(x) if x is not None else None for x in (cache.k, cache.v, cache.ks, cache.vs)]
    if in_place:
        q = q.contiguous()
    q0 = q.clone()
    got = fm.paged_append(k, v, cache.k, cache.v, cache.table, i32(start), counts=None if counts is None else i32(counts),
                          q=q if with_q else None, cos=cos, sin=sin, interleaved=interleaved,
                          positions=None if positions is None else i32(positions), q_out=q if in_place else None,
                          **cache.kw)
    want = [None if x is None else x.copy() for x in before]
    half = [np.full(x.shape, False) if x is not None else None for x in before]
    table = cache.table.cpu().numpy()
    for b in range(B):
        for i in range(N):
            if with_q and i >= real[b]:
                assert (got[b, i] == 0).all()
            if i >= real[b]:
                continue
            p = start[b] + i
            r = p if positions is None else positions[b][i]
            kx, vx, qx = f64(k[b, i]), f64(v[b, i]), f64(q0[b, i])
            kr, qr = kx, qx
            if rot:
                c, s = f64(cos[r]), f64(sin[r])
                kr, qr = ref.rotate(kx, c, s, interleaved), ref.rotate(qx, c, s, interleaved)
            if with_q:
                # products and sum in fp32 (2^-23 of |x1| + |x2| <= 2^-22 max |x|), then one rounding
                tol = HALF_BF16 * np.abs(qr) + 2.0 ** -21 * np.abs(qx).max(-1, keepdims=True)
                assert (np.abs(f64(got[b, i]) - qr) <= tol).all()
            page_, slot = table[b, p // page], p % page
            if bits == 16:
                tol = HALF_BF16 * np.abs(kr) + 2.0 ** -21 * np.abs(kx).max(-1, keepdims=True)
                assert (np.abs(f64(cache.k[page_, :, slot]) - kr) <= tol).all()
                want[0][page_, :, slot] = f64(cache.k[page_, :, slot])
                want[1][page_, :, slot] = vx
            else:
                for at, row in ((0, bf16(kr)), (1, vx)):
                    code, scale, lo = ref.quantise(row)
                    want[at][page_, :, slot] = code[:, 0::2] + 16 * code[:, 1::2]
                    want[2 + at][page_, :, slot] = np.stack([scale, lo], -1)
    for name, x, y in zip(("k", "v", "k_scales", "v_scales"), (cache.k, cache.v, cache.ks, cache.vs), want):
        if x is not None:
            assert np.array_equal(f64(x), y), name  # codes and scales exactly; other slots as they were
    if with_q:
        assert got.is_contiguous() and (not in_place or got is q)


@pytest.mark.parametrize("bits", [16, 4])
@pytest.mark.parametrize("B,N,Hq,Hkv,d,page,start,rot,inter", [
    (1, 1, 1, 1, 64, 16, [0], 64, False),
    (3, 1, 8, 2, 128, 16, [15, 16, 700], 128, False),
    (2, 37, 4, 4, 64, 32, [0, 31], 32, True),
    (1, 130, 6, 2, 128, 64, [63], 128, True),
    (2, 9, 3, 1, 128, 128, [5, 250], 64, False),
    (1, 33, 2, 16, 64, 256, [250], 48, False),
    (2, 5, 2, 1, 128, 16, [3, 14], 16, True),
    (2, 5, 2, 1, 128, 16, [3, 14], 0, False),
])
def test_append(bits, B, N, Hq, Hkv, d, page, start, rot, inter):
    check_append(bits, B, N, Hq, Hkv, d, page, start, rot, inter)


@pytest.mark.parametrize("bits", [16, 4])
def test_append_padded_batch_positions_and_in_place(bits):
    check_append(bits, 4, 20, 4, 2, 128, 16, [0, 7, 100, 31], 128, counts=[20, 0, 1, 13])
    check_append(bits, 2, 12, 4, 2, 64, 16, [40, 3], 64, positions=[[5] * 6 + list(range(6)), list(range(2988, 3000))])
    check_append(bits, 2, 12, 4, 2, 64, 16, [40, 3], 64, in_place=True, counts=[12, 4])
    check_append(bits, 2, 12, 4, 2, 64, 16, [40, 3], 64, with_q=False)


def test_append_many_rows_4bit_codes_are_the_nearest():
    """65536 rows of keys, rotated: every code equals the fp64 definition's."""
    check_append(4, 1, 2048, 1, 16, 64, 256, [0], 64, seed=77)


def test_append_4bit_special_rows():
    """Equal values, zeros, tiny and huge spreads, values on the middle of two codes; NaN and infinities read
    back as NaN in their row alone."""
    d, rows = 64, []
    rows.append(np.full(d, 1.5))
    rows.append(np.zeros(d))
    rows.append(np.linspace(-1, 1, d) * 2.0 ** -126)
    rows.append(np.linspace(-1, 1, d) * 2.0 ** -120)
    rows.append(np.linspace(-1, 1, d) * 2.0 ** 126)
    rows.append(np.arange(d) % 16 * 1.0)
    rows.append(np.where(np.arange(d) < 16, np.arange(d) * 2.0, np.arange(d) % 31))  # scale 2: odd values are ties
    rows.append(np.where(np.arange(d) % 2 == 0, -1.0, 2.0 ** -30))
    for bad in (np.nan, np.inf, -np.inf):
        x = np.linspace(-2, 3, d)
        x[11] = bad
        rows.append(x)
    x = np.linspace(-1, 1, d) * 3e38
    rows.append(x)
    n = len(rows)
    v = torch.from_numpy(np.stack(rows)).bfloat16().reshape(1, n, 1, d).cuda()
    cache = Cache(5, [n], 1, d, 16, 4).cuda()
    fm.paged_append(v, v, cache.k, cache.v, cache.table, i32([0]), **cache.kw)
    for t, s in ((cache.k, cache.ks), (cache.v, cache.vs)):
        for j in range(n):
            code, sc = f64(t[int(cache.table[0, 0]), 0, j]), f64(s[int(cache.table[0, 0]), 0, j])
            if j >= 8:
                assert np.isnan(sc).all(), j
                continue
            want, scale, lo = ref.quantise(f64(v[0, j, 0]))
            assert np.array_equal(code, want[0::2] + 16 * want[1::2]), j
            assert sc[0] == scale and sc[1] == lo
    k, _ = fm.paged_gather(cache.k, cache.v, cache.table, i32([n]), n, **cache.kw)
    assert torch.isnan(k[0, 8:]).all() and not torch.isnan(k[0, :8]).any()


def test_append_bad_positions_are_reported_and_left_out():
    cache = Cache(6, [40, 40], 1, 64, 16, 16).cuda()
    k = torch.randn(2, 4, 1, 64, device="cuda").bfloat16()
    q = torch.randn(2, 4, 2, 64, device="cuda").bfloat16()
    cos, sin = tables(41, 64)
    before = cache.k.clone()

    def run(start, table=None, **kw):
        kp, vp = cache.k.clone(), cache.v.clone()
        out = fm.paged_append(k, k, kp, vp, cache.table if table is None else table, i32(start), q=q, cos=cos, sin=sin, **kw)
        return kp, out

    good, _ = run([10, 20])
    assert fm.get_status() == 0 and not torch.equal(good, before)
    kp, out = run([46, -4])  # past the table's 48 positions, and in front of the first
    assert fm.get_status() == -9
    assert torch.equal(kp, before)  # 46 and 47 have no rotation angles either
    assert (out == 0).all()
    t = cache.table.clone()
    t[0, 0] = 10 ** 6
    kp, out = run([10, 20], t)
    assert fm.get_status() == -9
    want = good.clone()
    want[int(cache.table[0, 0]), :, 10:14] = before[int(cache.table[0, 0]), :, 10:14]
    assert torch.equal(kp, want)
    run([10, 20], positions=i32([[0, 1, 2, 3], [0, 1, 2, 41]]))
    assert fm.get_status() == -9
    run([10, 20], counts=i32([5, 1]))
    assert fm.get_status() == -9
    run([2 ** 31 - 2, 20])
    assert fm.get_status() == -9


def test_append_unaligned_views_are_refused():
    cache = Cache(6, [40], 1, 64, 16, 16).cuda()
    k = torch.zeros(1, 4, 1, 72, device="cuda").bfloat16()
    with pytest.raises(ValueError, match="16-byte"):
        fm.paged_append(k[..., 4:68], k[..., 4:68], cache.k, cache.v, cache.table, i32([0]))
    fm.paged_append(k[..., 8:], k[..., 8:], cache.k, cache.v, cache.table, i32([0]))


# ---------------------------------------------------------------------------
# gather
# ---------------------------------------------------------------------------
@pytest.mark.parametrize("bits", [16, 4])
@pytest.mark.parametrize("lens,N,Hkv,d,page", [
    ([1], 1, 1, 64, 16), ([0, 33, 16, 100], 100, 2, 128, 32), ([50, 20], 17, 3, 64, 16), ([700], 900, 1, 128, 256),
    ([5], 0, 2, 64, 16),
])
def test_gather(bits, lens, N, Hkv, d, page):
    cache = Cache(41, lens, Hkv, d, page, bits).cuda()
    k, v = fm.paged_gather(cache.k, cache.v, cache.table, i32(lens), N, **cache.kw)
    for b, n in enumerate(lens):
        m = min(n, N)
        for got, want in zip((k, v), cache.dense(b, m)):
            assert np.array_equal(f64(got[b, :m]), bf16(want))  # one rounding, the same
            assert (got[b, m:] == 0).all()


def test_gather_bad_entry_and_length():
    cache = Cache(42, [40], 1, 64, 16, 16).cuda()
    k0, _ = fm.paged_gather(cache.k, cache.v, cache.table, i32([40]), 40)
    t = cache.table.clone()
    t[0, 1] = -1
    k, _ = fm.paged_gather(cache.k, cache.v, t, i32([40]), 40)
    assert fm.get_status() == -9
    k0[0, 16:32] = 0
    assert torch.equal(k, k0)
    k, _ = fm.paged_gather(cache.k, cache.v, cache.table, i32([-5]), 40)
    assert fm.get_status() == -9 and (k == 0).all()
    k, _ = fm.paged_gather(cache.k, cache.v, cache.table, i32([10 ** 9]), 60)
    assert fm.get_status() == -9 and (k[0, 48:] == 0).all()


# ---------------------------------------------------------------------------
# together
# ---------------------------------------------------------------------------
@pytest.mark.parametrize("bits", [16, 4])
def test_serving_run(bits):
    """A prompt of documents is appended (rotation restarting at each), a second chunk attends to it through
    gather and the dense forward, then single tokens are appended and attended in a captured graph replayed
    with growing lengths.  Every row is compared with the fp64 attention over the cache's own values."""
    B, Hq, Hkv, d, page, n0, n1, steps = 2, 4, 2, 64, 16, 75, 29, 6
    total = n0 + n1 + steps
    rng = np.random.default_rng(9)
    cache = Cache(51, [total] * B, Hkv, d, page, bits).cuda()
    vec_np = np.stack([wl.causal_document_vectors([40, total - 40]), wl.causal_document_vectors([60, total - 60])], 1)
    vec = [torch.from_numpy(np.ascontiguousarray(x[:, None])).cuda() for x in vec_np]
    rope = np.stack([np.r_[np.arange(40), np.arange(total - 40)], np.r_[np.arange(60), np.arange(total - 60)]])
    qkv = torch.from_numpy(rng.standard_normal((B, total, Hq + 2 * Hkv, d))).bfloat16().cuda()
    cos, sin = tables(total, d)

    def append(a, n, lens):
        x = qkv[:, a:a + n]
        return fm.paged_append(x[:, :, Hq:Hq + Hkv], x[:, :, Hq + Hkv:], cache.k, cache.v, cache.table, lens,
                               q=x[:, :, :Hq], cos=cos, sin=sin, positions=i32(rope[:, a:a + n]), **cache.kw)

    def against(o, lse, q, a, n):
        ro, rl, to, tl = ref.attention(q, cache, [a + n] * B, vec)
        # the dense forward rounds the gathered 4-bit values to bf16 and its parity bound is 2e-2
        assert (np.abs(f64(o) - ro) <= to).all() and (np.abs(f64(lse) - rl) <= tl).all()

    q0 = append(0, n0, i32([0, 0]))
    o, lse = fm.paged_attention(q0, cache.k, cache.v, cache.table, i32([n0] * B), *vec, **cache.kw)
    against(o, lse, q0, 0, n0)
    # the chunk: its rows through the dense forward on gathered pages, masks cut to its rows
    q1 = append(n0, n1, i32([n0, n0]))
    k, v = fm.paged_gather(cache.k, cache.v, cache.table, i32([n0 + n1] * B), n0 + n1, **cache.kw)
    cut = [fm.localize(x[..., :n0 + n1].contiguous(), n0, n0 + n1) for x in vec]
    o, lse = fm.fwd(q1, k, v, *cut)
    po, pl = fm.paged_attention(q1, cache.k, cache.v, cache.table, i32([n0 + n1] * B), *vec, **cache.kw)
    assert (o.double() - po.double()).abs().max() <= 2e-2 and (lse - pl).abs().max() <= (1e-3 if bits == 16 else 2e-2)
    against(po, pl, q1, n0, n1)
    # single tokens in a graph: start and lens live on the device and move between replays
    start, lens = i32([n0 + n1] * B), i32([n0 + n1 + 1] * B)
    x = qkv[:, n0 + n1:n0 + n1 + 1].clone()
    pos = i32(rope[:, n0 + n1:n0 + n1 + 1])

    def step():
        q = fm.paged_append(x[:, :, Hq:Hq + Hkv], x[:, :, Hq + Hkv:], cache.k, cache.v, cache.table, start,
                            q=x[:, :, :Hq], cos=cos, sin=sin, positions=pos, **cache.kw)
        return (q,) + fm.paged_attention(q, cache.k, cache.v, cache.table, lens, *vec, **cache.kw)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        q, o, lse = step()
    for t in range(steps):
        a = n0 + n1 + t
        x.copy_(qkv[:, a:a + 1])
        pos.copy_(i32(rope[:, a:a + 1]))
        start.fill_(a)
        lens.fill_(a + 1)
        graph.replay()
        against(o, lse, q, a, 1)


@pytest.mark.parametrize("bits", [16, 4])
def test_two_streams_and_graphs_share_nothing(bits):
    """Calls overlapping on two streams, and two captured graphs replayed together, give the bits of single calls."""
    sets = []
    for s, lens in ((1, [3000, 50, 0]), (2, [10, 2100, 999])):
        cache, q = Cache(60 + s, lens, 2, 128, 64, bits).cuda(), case_q(3, 1, 8, 128, s)
        n = i32(lens)
        sets.append((q, cache, n, fm.paged_attention(q, cache.k, cache.v, cache.table, n, **cache.kw)))
    streams, graphs = [torch.cuda.Stream() for _ in sets], []
    torch.cuda.synchronize()
    for _ in range(20):
        outs = []
        for st, (q, c, n, _) in zip(streams, sets):
            with torch.cuda.stream(st):
                outs.append(fm.paged_attention(q, c.k, c.v, c.table, n, **c.kw))
        torch.cuda.synchronize()
        for (o, l), (_, _, _, (ro, rl)) in zip(outs, sets):
            assert torch.equal(o, ro) and torch.equal(l, rl)
    pool = torch.cuda.graph_pool_handle()
    for q, c, n, _ in sets:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, pool=pool):
            out = fm.paged_attention(q, c.k, c.v, c.table, n, **c.kw)
        graphs.append((g, out))
    for _ in range(5):
        for g, _ in graphs:
            g.replay()
    torch.cuda.synchronize()
    for (_, (o, l)), (_, _, _, (ro, rl)) in zip(graphs[::-1], sets[::-1]):
        assert torch.equal(o, ro) and torch.equal(l, rl)
