"""Paged key/value cache on the GPU, at values, outputs and calls that tests/test_gpu_paged.py does not reach: codes
whose exact quotient lies beside the middle of two codes by less than fp32 sees, outputs inside the caller's buffers,
offsets past 31 bits, graphs replayed at the same time, and the cap on CTAs."""
from fractions import Fraction

import numpy as np
import pytest
import torch

import column_sparse_masked_b200 as fm

import _paged as ref
from _paged import Cache, bf16, f64

pytestmark = pytest.mark.gpu


def i32(x):
    return torch.tensor(np.asarray(x), dtype=torch.int32).cuda()


@pytest.fixture(autouse=True)
def clean_status():
    fm.get_status()
    yield
    assert fm.get_status() == 0


# ---------------------------------------------------------------------------
# append, 4 bits: the code decision
# ---------------------------------------------------------------------------
def nearest_code(x, lo, scale):
    """The integer nearest to (x - lo) / scale, ties to even, in rational arithmetic."""
    return min(max(round((Fraction(x) - Fraction(lo)) / Fraction(scale)), 0), 15)  # Fraction: ties to even


def rows_beside_the_middle(d):
    """Rows of bf16 values with quotients on the middle of two codes but for a term that a sum in fp32 loses: a
    minimum of (k + 1/2) steps and values near 0, or a minimum near 0 and values of (k + 1/2) steps."""
    rows = []
    for a in (-60, -3, 0, 1, 40):
        step = 2.0 ** a
        tiny = [0.0] + [s * m * step * 2.0 ** -e for e in (8, 20, 23, 24, 25, 26, 30, 33, 60) for s in (1, -1)
                        for m in (1.0, 1.5)]
        for k in range(16):  # 0 lies k + 1/2 (or k) steps above the minimum
            for part in (0.5, 0.0):
                lo = -(k + part) * step
                x = [lo, lo + 15 * step] + tiny
                rows.append(x + [0.0] * (d - len(x)))
        odd = [(k + 0.5) * step for k in range(15)]
        for t in tiny:
            x = [t if t < 0 else min(t, 0.25 * step), 15 * step] + odd + [k * step for k in range(1, 15)]
            rows.append(x + [step] * (d - len(x)))
    return bf16(np.array(rows))


@pytest.mark.parametrize("d", [64, 128])
def test_codes_beside_the_middle_of_two(d):
    """Every code is the nearest one for the row's stored scale and minimum, ties to even, in rational arithmetic."""
    x = rows_beside_the_middle(d)
    x = np.concatenate([x, x[:, ::-1]])
    n = len(x)
    cache = Cache(71, [n], 1, d, 64, 4).cuda()
    t = torch.from_numpy(x).bfloat16().reshape(1, n, 1, d).cuda()
    assert np.array_equal(f64(t).reshape(n, d), x)
    fm.paged_append(t, t, cache.k, cache.v, cache.table, i32([0]), **cache.kw)
    page = cache.table[0].cpu().numpy()[np.arange(n) // 64]
    for codes, scales in ((cache.k, cache.ks), (cache.v, cache.vs)):
        c, s = codes.cpu().numpy()[page, 0, np.arange(n) % 64], f64(scales)[page, 0, np.arange(n) % 64]
        got = np.stack([c & 15, c >> 4], -1).reshape(n, d)
        _, scale, lo = ref.quantise(x)
        assert np.array_equal(s, np.stack([scale, lo], -1))
        want = np.array([[nearest_code(y, lo[i], scale[i]) for y in x[i]] for i in range(n)])
        assert np.array_equal(got, want)


# ---------------------------------------------------------------------------
# gather: outputs inside the caller's buffers
# ---------------------------------------------------------------------------
@pytest.mark.parametrize("bits", [16, 4])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("at_k,at_v", [(8, 16), (16, 8), (8, 24), (0, 0)])
def test_gather_into_16_byte_aligned_outputs(bits, d, at_k, at_v):
    """Outputs anywhere in a buffer, as long as they are 16-byte aligned; nothing beside them is written."""
    lens, N, Hkv = [37, 0, 64], 50, 3
    cache = Cache(72, lens, Hkv, d, 16, bits).cuda()
    want = fm.paged_gather(cache.k, cache.v, cache.table, i32(lens), N, **cache.kw)
    size = want[0].numel()
    buffers = [torch.full((size + 48,), 7.0, dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    out = tuple(x[a:a + size].view(want[0].shape) for x, a in zip(buffers, (at_k, at_v)))
    got = fm.paged_gather(cache.k, cache.v, cache.table, i32(lens), N, out=out, **cache.kw)
    assert got[0] is out[0] and got[1] is out[1]
    for x, a, w in zip(buffers, (at_k, at_v), want):
        assert torch.equal(x[a:a + size].view(w.shape), w)
        assert (x[:a] == 7).all() and (x[a + size:] == 7).all()


def test_gather_refuses_outputs_off_the_16_byte_grid():
    cache = Cache(72, [20], 1, 64, 16, 16).cuda()
    x = torch.zeros(2, 20 * 64 + 8, dtype=torch.bfloat16, device="cuda")
    with pytest.raises(fm.FlashMaskError, match="align"):
        fm.paged_gather(cache.k, cache.v, cache.table, i32([20]), 20,
                        out=(x[0, 4:4 + 20 * 64].view(1, 20, 1, 64), x[1, :20 * 64].view(1, 20, 1, 64)))


# ---------------------------------------------------------------------------
# append: offsets that pass 32 bits
# ---------------------------------------------------------------------------
def test_append_q_rows_whose_offsets_pass_31_bits():
    """A row of more than 2^24 q-heads of 128: values beyond the 2^31st of q_out are where they belong, and those in
    front of the buffer's start (where a wrapped offset would point) are left alone."""
    Hq, d = (1 << 24) + 5, 128
    cache = Cache(73, [1], 1, d, 16, 16).cuda()
    row = torch.randn(1, 1, 1, d, device="cuda").bfloat16()
    lead = 1 << 16
    buf = torch.full((lead + Hq * d,), 7.0, dtype=torch.bfloat16, device="cuda")
    out = buf[lead:].view(1, 1, Hq, d)
    fm.paged_append(row, row, cache.k, cache.v, cache.table, i32([0]), q=row.expand(1, 1, Hq, d), q_out=out)
    assert (buf[:lead] == 7).all()
    for a in range(0, Hq, 1 << 22):
        assert torch.equal(out[0, 0, a:a + (1 << 22)], row[0, 0].expand(min(1 << 22, Hq - a), d)), a


# ---------------------------------------------------------------------------
# attention: graphs at once, and the cap on CTAs
# ---------------------------------------------------------------------------
def sequences(seed, lens, bits, Hkv=2, d=128, width=None):
    cache = Cache(seed, lens, Hkv, d, 64, bits, width=width).cuda()
    g = torch.Generator().manual_seed(seed)
    return cache, torch.randn(len(lens), 1, 4 * Hkv, d, generator=g).bfloat16().cuda(), i32(lens)


def window(B, n, size):
    """Causal windows of `size` keys, one mask head."""
    j = torch.arange(n, dtype=torch.int32, device="cuda").expand(B, 1, n)
    return [(j + size).contiguous(), torch.full_like(j, n + 1).contiguous(), None, None]


@pytest.mark.parametrize("bits", [16, 4])
@pytest.mark.parametrize("masked", [False, True])
def test_graphs_on_their_own_streams_share_nothing(bits, masked):
    """Two graphs with a memory pool each, replayed at the same time on two streams, give the bits of single calls in
    every round."""
    sets = []
    for seed, lens in ((81, [3000, 50, 0]), (82, [10, 2100, 999])):
        cache, q, n = sequences(seed, lens, bits)
        vec = window(3, max(lens), 700) if masked else [None] * 4
        call = (lambda q=q, c=cache, n=n, vec=vec: fm.paged_attention(q, c.k, c.v, c.table, n, *vec, **c.kw))
        sets.append((call, call(), torch.cuda.Stream(), torch.cuda.CUDAGraph()))
    torch.cuda.synchronize()
    outs = []
    for call, _, _, graph in sets:
        with torch.cuda.graph(graph):
            outs.append(call())
    for _ in range(20):
        for o, lse in outs:
            o.fill_(7), lse.fill_(7)
        torch.cuda.synchronize()
        for _, _, stream, graph in sets:
            with torch.cuda.stream(stream):
                for _ in range(4):
                    graph.replay()
        torch.cuda.synchronize()
        for (o, lse), (_, (ro, rl), _, _) in zip(outs, sets):
            assert torch.equal(o, ro) and torch.equal(lse, rl)


@pytest.mark.parametrize("bits", [16, 4])
@pytest.mark.parametrize("lens,width,B,same", [([300, 90], None, 2, True), ([200, 17] * 80, None, 160, True),
                                               ([5000, 300], 90, 2, False)])
def test_the_cap_on_ctas_changes_the_order_of_sums_at_most(bits, lens, width, B, same):
    """Items of one CTA and whole items of a warp give the same bits under any cap; items that are cut are cut
    elsewhere, and their parts are joined in fp32."""
    cache, q, n = sequences(83, lens, bits, width=width)
    o, lse = fm.paged_attention(q, cache.k, cache.v, cache.table, n, **cache.kw)
    try:
        for cap in (1, 3, 40):
            fm.set_max_ctas(cap)
            o2, l2 = fm.paged_attention(q, cache.k, cache.v, cache.table, n, **cache.kw)
            if same:
                assert torch.equal(o, o2) and torch.equal(lse, l2)
            # weights are rounded to bf16 against another running maximum, 2^-8 each on either side, and the
            # result once more: 2^-8 (2 sum w |v| + 2 |o|), with |v| <= 5.5 (normal values, or -3 + 0.5 x 15)
            assert (o.double() - o2.double()).abs().max() <= 4 * 2.0 ** -8 * 5.5
            # fp32: 2^-20 covers exp2, log2 and the sums
            assert ((lse.double() - l2.double()).abs() <= 2.0 ** -19 * (1 + lse.double().abs())).all()
    finally:
        fm.set_max_ctas(0)
