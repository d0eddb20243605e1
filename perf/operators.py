"""Cases and plain forms of the paged-cache operators.

Serving a model that was trained with column-sparse masked attention needs a
key/value cache in pages, held in bf16 or in 4 bits: new keys are rotated to
their positions and appended, rows of new tokens attend to the pages through
the same column-wise mask vectors, and a long chunk's keys are gathered back
into the dense layout that the forward takes.

  append     q, k [B, N, H, d] rotated by cos/sin tables, k and v written into
             their pages (bf16, or codes 0..15 with a scale and a minimum)
  attention  o, lse of rows [B, Nq, Hq, d] over the pages
  gather     pages as dense k, v [B, N, Hkv, d] bf16

Where `own` is true, `run` calls the package; where it is false, the same is
computed with elementary torch operations.
"""
import math
import random

import numpy as np
import torch

own = False

F32, F64, BF16 = torch.float32, torch.float64, torch.bfloat16


# ---------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------
def _append(name, bits, B, N, Hq, Hkv, d, page, past, rot, inter, ragged, docs):
    return {"name": name, "op": "append", "bits": bits, "B": B, "N": N, "Hq": Hq, "Hkv": Hkv, "d": d, "page": page,
            "past": past, "rot": rot, "interleaved": inter, "ragged": ragged, "docs": docs}


def _attention(name, bits, B, Nq, Hq, Hkv, d, page, lo, hi, mask, Hm=1):
    return {"name": name, "op": "attention", "bits": bits, "B": B, "Nq": Nq, "Hq": Hq, "Hkv": Hkv, "d": d,
            "page": page, "lo": lo, "hi": hi, "mask": mask, "Hm": Hm}


def _gather(name, bits, B, Hkv, d, page, lo, hi):
    return {"name": name, "op": "gather", "bits": bits, "B": B, "Hkv": Hkv, "d": d, "page": page, "lo": lo, "hi": hi}


def listed():
    return [
        # one decode step of 64 sequences: one new token each, at ragged positions
        _append("append_decode64", 16, 64, 1, 32, 8, 128, 64, 1000, 128, False, False, False),
        # a prompt of packed documents: rotation positions restart at each document
        _append("append_prompt8k", 16, 1, 8192, 32, 8, 128, 64, 0, 128, False, False, True),
        # one decode step into a 4-bit cache, half of the head rotated, pairs side by side
        _append("append4_decode37", 4, 37, 1, 16, 4, 64, 16, 333, 32, True, False, False),
        # chunks of 9 prompts of different lengths, padded to one batch, into a 4-bit cache
        _append("append4_prompt_ragged", 4, 9, 1021, 32, 8, 128, 32, 77, 128, False, True, False),
        # dense keys and values for a long chunk's forward, out of a bf16 cache of ragged sequences
        _gather("gather_ragged", 16, 5, 8, 128, 64, 100, 4001),
        # the same for one 32K sequence of a 4-bit cache
        _gather("gather4_32k", 4, 1, 16, 128, 128, 32768, 32768),
        # the smallest step: one row, two heads, 256 keys
        _attention("decode_tiny", 16, 1, 1, 2, 2, 64, 16, 256, 256, "none"),
        # a decode batch of 64 sequences of ragged lengths up to 8K
        _attention("decode_batch64", 16, 64, 1, 32, 8, 128, 64, 256, 8192, "none"),
        # one row at the end of 128K tokens of documents with 30 % of the key tiles dropped
        _attention("decode_docs128k", 16, 1, 1, 32, 8, 128, 128, 131072, 131072, "doc_blocksparse"),
        # a run of 5 new rows (drafted tokens) after a shared question with sibling answers
        _attention("verify_sharequestion32k", 16, 1, 5, 16, 16, 128, 64, 32768, 32768, "share_question"),
        # the decode batch over a cache held in 4 bits
        _attention("decode4_batch64", 4, 64, 1, 32, 8, 128, 64, 256, 8192, "none"),
        # prefix and sliding window, two 64K sequences, 4 bits
        _attention("decode4_prefixwindow64k", 4, 2, 1, 16, 16, 128, 64, 65536, 65536, "prefix_window"),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["append", "append", "attention", "attention", "attention", "gather"])
    bits = rng.choice([16, 4])
    d = rng.choice([64, 128, 128])
    page = rng.choice([16, 32, 64, 128])
    Hkv = rng.choice([1, 2, 4, 8, 16])
    G = rng.choice([1, 2, 3, 4, 8])
    B = _log_int(rng, 1, 64)
    if op == "append":
        N = _log_int(rng, 1, max(1, min(8192, 8192 * 48 // ((G + 2) * Hkv)) // B))
        rot = rng.choice([d, d, d // 2])
        c = _append("", bits, B, N, G * Hkv, Hkv, d, page, rng.randrange(0, 700), rot, rng.random() < 0.4,
                    rng.random() < 0.5, rng.random() < 0.3)
    elif op == "gather":
        hi = _log_int(rng, 16, max(17, (1 << 19) // (B * Hkv)))
        c = _gather("", bits, B, Hkv, d, page, max(1, hi // rng.randrange(1, 40)), hi)
    else:
        hi = _log_int(rng, 16, min(131072, 1100000 // (B * Hkv)))
        lo = max(1, hi // rng.randrange(1, 40))
        mask = rng.choice(["none", "none", "prefix_window", "doc_blocksparse", "share_question", "random"])
        Hm = G * Hkv if mask == "random" and B * hi * G * Hkv <= 1 << 21 and rng.random() < 0.7 else 1
        c = _attention("", bits, B, rng.choice([1, 1, 1, 2, 3, 5, 8, 16]), G * Hkv, Hkv, d, page, lo, hi, mask, Hm)
        if B * hi * G * Hkv * c["Nq"] > 1 << 26:
            c["Nq"] = 1
    del c["name"]
    return c


# ---------------------------------------------------------------------------
# sizes and masks that follow from the case alone
# ---------------------------------------------------------------------------
def _rng(case):
    return np.random.default_rng(sum((i + 1) * int(v) for i, v in enumerate(
        case.get(n, 0) for n in ("B", "N", "Nq", "Hq", "Hkv", "d", "page", "lo", "hi", "past", "bits"))))


def _lens(case):
    """Cached tokens of each sequence, spread over [lo, hi] by their logarithm; the first is hi."""
    r = np.exp(_rng(case).uniform(math.log(case["lo"]), math.log(case["hi"] + 0.5), case["B"])).astype(np.int64)
    r = np.clip(r, case["lo"], case["hi"])
    r[0] = case["hi"]
    return r


def _new(case):
    """(start, counts) of an append: tokens cached before, and real tokens among the N."""
    r = _rng(case)
    start = r.integers(0, case["past"] + 1, case["B"])
    counts = r.integers(1, case["N"] + 1, case["B"]) if case["ragged"] else np.full(case["B"], case["N"])
    return start, counts


def _mask_vectors(case):
    """[4, B, Hm, hi] int32 column vectors (LTS, LTE, UTS, UTE), or None."""
    n, B, Hm, kind = case["hi"], case["B"], case["Hm"], case["mask"]
    if kind == "none":
        return None
    r = _rng(case)
    j = np.arange(n)
    v = np.zeros((4, B, Hm, n), np.int64)
    v[0], v[1], v[3] = n + case["Nq"], n + case["Nq"], j  # nothing hidden below, causal above
    if kind == "random":
        a = np.sort(r.integers(-2, n + 3, (4, B, Hm, n)).reshape(2, 2, B, Hm, n), axis=1)
        return a.reshape(4, B, Hm, n).astype(np.int32)
    if kind == "prefix_window":
        prefix, window = min(2048, n // 8), min(4096, n // 4 + 1)
        v[3][..., :prefix] = 0
        v[0] = np.minimum(j + window, n + case["Nq"])
    else:
        length = r.integers(max(1, n // 128), max(1, n // 4) + 1, 128)  # documents
        cuts = np.unique(np.concatenate([[0, n], np.minimum(np.cumsum(length), n)]))
        if kind == "share_question":  # the last segment: a question, then answers that do not see one another
            q_end = max(1, n // 2)
            cuts = np.unique(np.concatenate([[0, n], q_end + r.integers(0, n - q_end + 1, 4)]))
        end = cuts[np.searchsorted(cuts, j, side="right")]
        end[end == n] = n + case["Nq"]
        if kind == "share_question":
            end[:q_end] = n + case["Nq"]
        v[0] = end
        if kind == "doc_blocksparse":
            drop = r.random(-(-n // 128)) < 0.3
            v[0][..., drop[j // 128] & (j < n - 128)] = 0
    return v.astype(np.int32)


def _visible(case):
    """(keys that some row of their sequence sees, summed over sequences; pairs of a row and a key of one head)."""
    lens, vec = _lens(case), _mask_vectors(case)
    j = np.arange(case["hi"])
    keys = pairs = 0
    for b in range(case["B"]):
        some = np.zeros(case["hi"], bool)
        for i in range(case["Nq"]):
            p = lens[b] - case["Nq"] + i
            see = np.broadcast_to((j < lens[b]) & (j <= p), (case["Hm"], case["hi"]))
            if vec is not None:
                a, e, f, g = vec[:, b]
                see = see & ~(((a <= p) & (p < e)) | ((f <= p) & (p < g)))
            pairs += int(see.sum()) * (case["Hq"] // case["Hm"])
            some |= see.any(0)
        keys += int(some.sum())
    return keys, pairs


def _token_bytes(case):
    """Bytes of one token of one KV head in the cache, keys and values."""
    return 2 * (2 * case["d"] if case["bits"] == 16 else case["d"] // 2 + 4)


def work(case):
    d = case["d"]
    if case["op"] == "append":
        T = int(_new(case)[1].sum())
        rows = T * (case["Hq"] + 2 * case["Hkv"])
        table = min(T, case["N"]) * case["rot"] * 4
        b = rows * d * 2 + T * case["Hq"] * d * 2 + T * case["Hkv"] * _token_bytes(case) + table
        if case["bits"] == 4:  # the values come back dense as well
            n = int((_new(case)[0] + _new(case)[1]).sum())
            b += n * case["Hkv"] * (_token_bytes(case) + 4 * d)
        return {"bytes": b, "flops": 3 * rows * d}
    if case["op"] == "gather":
        n = int(_lens(case).sum())
        return {"bytes": n * case["Hkv"] * _token_bytes(case) + case["B"] * case["hi"] * case["Hkv"] * 4 * d,
                "flops": 2 * n * case["Hkv"] * d}
    keys, pairs = _visible(case)
    rows = case["B"] * case["Nq"] * case["Hq"]
    b = keys * case["Hkv"] * _token_bytes(case) + rows * (4 * d + 4)
    if case["mask"] != "none":
        b += 16 * case["Hm"] * int(_lens(case).sum())
    return {"bytes": b, "flops": 4 * d * pairs}


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------
def _randn(g, *shape):
    return torch.randn(*shape, generator=g, device="cuda", dtype=BF16)


def _pages(case, g, n_pages):
    """A cache of n_pages pages with data in every slot."""
    H, page, d = case["Hkv"], case["page"], case["d"]
    if case["bits"] == 16:
        return {"k_pages": _randn(g, n_pages, H, page, d), "v_pages": _randn(g, n_pages, H, page, d)}
    s = {}
    for n in ("k", "v"):
        s[n + "_pages"] = torch.randint(0, 256, (n_pages, H, page, d // 2), generator=g, device="cuda",
                                        dtype=torch.uint8)
        # least and largest value of a head's row of standard normal values
        end = 1.8 + 1.2 * torch.rand(n_pages, H, page, 2, generator=g, device="cuda", dtype=F32)
        s[n + "_scales"] = torch.stack([(end[..., 0] + end[..., 1]) / 15, -end[..., 1]], -1).to(BF16)
    return s


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    B, page, d = case["B"], case["page"], case["d"]
    if case["op"] == "append":
        start, counts = _new(case)
        lens = start + counts
    else:
        lens = _lens(case)
    width = -(-int(lens.max()) // page)
    # pages handed out in no order, as an allocator that has run for a while does
    n_pages = int((-(-lens // page)).sum()) + 3
    order = torch.randperm(n_pages, generator=g, device="cuda").to(torch.int32)
    used = -(-lens // page)
    at = np.cumsum(used) - used
    index = np.where(np.arange(width)[None] < used[:, None], at[:, None] + np.arange(width)[None], 0)
    s = _pages(case, g, n_pages)
    s["case"] = case
    s["table"] = order[torch.from_numpy(index).cuda()].contiguous()
    s["lens"] = torch.from_numpy(lens.astype(np.int32)).cuda()
    s["lens_host"] = lens
    if case["op"] == "append":
        N, T = case["N"], case["B"] * case["N"]
        s["qkv"] = _randn(g, B, N, case["Hq"] + 2 * case["Hkv"], d)  # one projection's output, split by views
        s["start"] = torch.from_numpy(start.astype(np.int32)).cuda()
        s["counts"] = torch.from_numpy(counts.astype(np.int32)).cuda() if case["ragged"] else None
        real = np.arange(N)[None] < counts[:, None]
        pos = start[:, None] + np.arange(N)[None]
        if case["docs"]:  # packed documents: the rotation starts again at each
            cut = np.maximum.accumulate(np.where(_rng(case).random((B, N)) < 3.0 / (N + 2), np.arange(N)[None], 0), 1)
            rope = np.arange(N)[None] - cut
            s["positions"] = torch.from_numpy(rope.astype(np.int32)).cuda()
        else:
            rope, s["positions"] = pos, None
        n_pos = int(max(pos.max(), rope.max())) + 1
        inv = 10000.0 ** (-np.arange(0, case["rot"], 2) / case["rot"])
        angle = torch.from_numpy(np.arange(n_pos)[:, None] * inv[None]).cuda()
        s["cos"], s["sin"] = angle.cos().to(F32), angle.sin().to(F32)
        # what a program without the operator would keep: where each real token goes
        s["token"] = torch.from_numpy(np.nonzero(real.reshape(T))[0]).cuda()
        b = np.nonzero(real)[0]
        s["slot_b"] = torch.from_numpy(b).cuda()
        s["slot_pos"] = torch.from_numpy(pos[real]).cuda()
        s["rope"] = torch.from_numpy(rope).cuda()
    elif case["op"] == "attention":
        s["q"] = _randn(g, B, case["Nq"], case["Hq"], d)
        vec = _mask_vectors(case)
        s["mask"] = [None] * 4 if vec is None else [torch.from_numpy(x).cuda() for x in vec]
    return s


# ---------------------------------------------------------------------------
# plain forms
# ---------------------------------------------------------------------------
def _rotate(x, cos, sin, interleaved):
    """x [.., H, d] with the first rot = 2 * cos.shape[-1] values rotated; cos, sin [.., 1, rot/2]."""
    r = cos.shape[-1]
    if interleaved:
        a, b = x[..., 0:2 * r:2], x[..., 1:2 * r:2]
        y = torch.stack([a * cos - b * sin, b * cos + a * sin], -1).flatten(-2)
    else:
        a, b = x[..., :r], x[..., r:2 * r]
        y = torch.cat([a * cos - b * sin, b * cos + a * sin], -1)
    return torch.cat([y, x[..., 2 * r:]], -1)


def _quantise(x):
    """Codes 0..15 packed in pairs and (scale, minimum) of the rows of x (bf16 values); in 64 bits, as a
    value next to the middle of two codes decides which."""
    x = x.to(F64)
    lo, hi = x.amin(-1, keepdim=True), x.amax(-1, keepdim=True)
    scale = ((hi - lo) / 15).to(F32).to(BF16)
    s = scale.to(F64)
    code = torch.where(s > 0, ((x - lo) / torch.where(s > 0, s, 1.0)).round().clamp(0, 15), 0.0).to(torch.uint8)
    return code[..., 0::2] | (code[..., 1::2] << 4), torch.cat([scale, lo.to(BF16)], -1)


def _values(codes, scales):
    """The values (32 bits) that packed codes stand for."""
    c = torch.stack([codes & 15, codes >> 4], -1).flatten(-2).to(F32)
    return scales[..., 1:2].to(F32) + scales[..., 0:1].to(F32) * c


def _dense(s, which, length):
    """Keys or values of the first `length` tokens, [B, length, Hkv, d] in 32 bits."""
    case = s["case"]
    j = torch.arange(length, device="cuda")
    page = s["table"][:, j // case["page"]].long()
    off = (j % case["page"])[None].expand_as(page)
    x = s[which + "_pages"][page, :, off]
    return x.to(F32) if case["bits"] == 16 else _values(x, s[which + "_scales"][page, :, off])


def _plain_gather(s, length):
    keep = torch.arange(length, device="cuda")[None] < s["lens"][:, None]
    return [torch.where(keep[..., None, None], _dense(s, n, length), 0.0).to(BF16) for n in ("k", "v")]


def _plain_append(s):
    case = s["case"]
    Hq, Hkv = case["Hq"], case["Hkv"]
    wide = F32 if case["bits"] == 16 else F64
    cos, sin = s["cos"][s["rope"]][:, :, None].to(wide), s["sin"][s["rope"]][:, :, None].to(wide)
    q = _rotate(s["qkv"][:, :, :Hq].to(wide), cos, sin, case["interleaved"]).to(F32).to(BF16)
    k = _rotate(s["qkv"][:, :, Hq:Hq + Hkv].to(wide), cos, sin, case["interleaved"]).to(F32).to(BF16)
    k, v = k.flatten(0, 1)[s["token"]], s["qkv"][:, :, Hq + Hkv:].flatten(0, 1)[s["token"]]
    page = s["table"][s["slot_b"], s["slot_pos"] // case["page"]].long()
    off = s["slot_pos"] % case["page"]
    if case["bits"] == 16:
        s["k_pages"][page, :, off] = k
        s["v_pages"][page, :, off] = v
    else:
        kc, ks = _quantise(k)
        vc, vs = _quantise(v)
        s["k_pages"][page, :, off], s["k_scales"][page, :, off] = kc, ks
        s["v_pages"][page, :, off], s["v_scales"][page, :, off] = vc, vs
    return q


def _plain_attention(s):
    case = s["case"]
    B, Nq, Hq, Hkv, d, n = (case[x] for x in ("B", "Nq", "Hq", "Hkv", "d", "hi"))
    k, v = _dense(s, "k", n).permute(0, 2, 1, 3), _dense(s, "v", n).permute(0, 2, 1, 3)
    q = s["q"].to(F32).permute(0, 2, 1, 3).reshape(B, Hkv, Hq // Hkv * Nq, d)
    x = (q @ k.transpose(-1, -2)).reshape(B, Hq, Nq, n) / math.sqrt(d)
    j = torch.arange(n, device="cuda")
    p = (s["lens"][:, None] - Nq + torch.arange(Nq, device="cuda")[None])[:, None, :, None]
    see = (j < s["lens"][:, None, None, None]) & (j <= p)
    if s["mask"][0] is not None:
        a, e, f, g = (m[:, :, None, :] for m in s["mask"])
        see = see & ~(((a <= p) & (p < e)) | ((f <= p) & (p < g)))
    x = torch.where(see, x, -math.inf)
    m = x.amax(-1, keepdim=True)
    m0 = torch.where(m == -math.inf, 0.0, m)
    w = torch.exp(x - m0)
    total = w.sum(-1, keepdim=True)
    o = w.reshape(B, Hkv, -1, n) @ torch.where((j < s["lens"][:, None])[:, None, :, None], v, 0.0)
    o = o.reshape(B, Hq, Nq, d) / torch.where(total > 0, total, 1.0)
    return o.permute(0, 2, 1, 3).to(BF16), (m0 + torch.log(total))[..., 0]


def run(s):
    case = s["case"]
    if own:
        return _run_own(s)
    if case["op"] == "attention":
        return _plain_attention(s)
    if case["op"] == "gather":
        return _plain_gather(s, case["hi"])
    q = _plain_append(s)
    if case["ragged"]:  # rows behind a sequence's last token hold nothing
        q = torch.where((torch.arange(case["N"], device="cuda")[None] < s["counts"][:, None])[..., None, None], q, 0)
    if case["bits"] == 16:
        return q, s["k_pages"], s["v_pages"]
    return [q] + _plain_gather(s, int(s["lens_host"].max())) + [s["k_scales"], s["v_scales"]]


def _run_own(s):
    import column_sparse_masked_b200 as fm

    case = s["case"]
    scales = {"k_scales": s.get("k_scales"), "v_scales": s.get("v_scales")}
    if case["op"] == "attention":
        lts, lte, uts, ute = s["mask"]
        return fm.paged_attention(s["q"], s["k_pages"], s["v_pages"], s["table"], s["lens"], lts, lte, uts, ute,
                                  **scales)
    if case["op"] == "gather":
        return fm.paged_gather(s["k_pages"], s["v_pages"], s["table"], s["lens"], case["hi"], **scales)
    Hq, Hkv = case["Hq"], case["Hkv"]
    qkv = s["qkv"]
    q = fm.paged_append(qkv[:, :, Hq:Hq + Hkv], qkv[:, :, Hq + Hkv:], s["k_pages"], s["v_pages"], s["table"],
                        s["start"], counts=s["counts"], q=qkv[:, :, :Hq], cos=s["cos"], sin=s["sin"],
                        positions=s["positions"], interleaved=case["interleaved"], **scales)
    if case["bits"] == 16:
        return q, s["k_pages"], s["v_pages"]
    k, v = fm.paged_gather(s["k_pages"], s["v_pages"], s["table"], s["lens"], int(s["lens_host"].max()), **scales)
    return q, k, v, s["k_scales"], s["v_scales"]


# ---------------------------------------------------------------------------
# the definitions in 64 bits
# ---------------------------------------------------------------------------
def _sequence(s, which, b, n):
    """Values of the first n tokens of sequence b, [n, Hkv, d] in 64 bits."""
    case = s["case"]
    ids = s["table"][b, : -(-n // case["page"])].long()
    x = s[which + "_pages"].index_select(0, ids).transpose(1, 2).reshape(-1, case["Hkv"], s[which + "_pages"].shape[-1])
    if case["bits"] == 16:
        return x[:n].double()
    sc = s[which + "_scales"].index_select(0, ids).transpose(1, 2).reshape(-1, case["Hkv"], 2)[:n].double()
    out = torch.empty(n, case["Hkv"], case["d"], dtype=F64, device="cuda")
    out[..., 0::2] = (x[:n] % 16).double()
    out[..., 1::2] = (x[:n] // 16).double()
    return out.mul_(sc[..., :1]).add_(sc[..., 1:])


def _exact_gather(s, n):
    out = []
    for which in ("k", "v"):
        t = torch.zeros(s["case"]["B"], n, s["case"]["Hkv"], s["case"]["d"], dtype=F64, device="cuda")
        for b, L in enumerate(s["lens_host"].tolist()):
            t[b, :L] = _sequence(s, which, b, L)
        out.append(t)
    return out


def _turn(x, s, b, count):
    """Rows 0..count of sequence b turned by their angles, as complex numbers."""
    case, r = s["case"], s["case"]["rot"] // 2
    at = s["rope"][b, :count]
    turn = torch.complex(s["cos"][at].double(), s["sin"][at].double())[:, None]
    y = x.double().clone()
    lo, hi = (slice(0, 2 * r, 2), slice(1, 2 * r, 2)) if case["interleaved"] else (slice(0, r), slice(r, 2 * r))
    z = torch.complex(y[..., lo].contiguous(), y[..., hi].contiguous()) * turn
    y[..., lo], y[..., hi] = z.real, z.imag
    return y


def _exact_append(s):
    case = s["case"]
    Hq, Hkv, page = case["Hq"], case["Hkv"], case["page"]
    start, counts = _new(case)
    q = torch.zeros(case["B"], case["N"], Hq, case["d"], dtype=F64, device="cuda")
    pages = {n: s[n + "_pages"].double() if case["bits"] == 16 else None for n in ("k", "v")}
    for b in range(case["B"]):
        a, c = int(start[b]), int(counts[b])
        x = s["qkv"][b, :c]
        q[b, :c] = _turn(x[:, :Hq], s, b, c)
        new = {"k": _turn(x[:, Hq:Hq + Hkv], s, b, c), "v": x[:, Hq + Hkv:].double()}
        pos = torch.arange(a, a + c, device="cuda")
        ids, off = s["table"][b].long()[pos // page], pos % page
        for n, y in new.items():
            if case["bits"] == 16:
                pages[n][ids, :, off] = y
                continue
            y = y.float().bfloat16().double()  # a 4-bit row is made from the bf16 row
            lo, hi = y.min(-1)[0], y.max(-1)[0]
            step = ((hi - lo) / 15).float().bfloat16()
            t = (y - lo[..., None]) / step.double().clamp_min(1e-300)[..., None]
            code = torch.floor(t)
            rest = t - code
            code += ((rest > 0.5) | ((rest == 0.5) & (code % 2 == 1))).double()
            code = code.clamp(0, 15) * (step.double() > 0)[..., None]
            s[n + "_pages"][ids, :, off] = (code[..., 0::2] + 16 * code[..., 1::2]).to(torch.uint8)
            s[n + "_scales"][ids, :, off] = torch.stack([step, lo.bfloat16()], -1)
    if case["bits"] == 16:
        return q, pages["k"], pages["v"]
    return [q] + _exact_gather(s, int(s["lens_host"].max())) + [s["k_scales"].double(), s["v_scales"].double()]


def _exact_attention(s):
    case = s["case"]
    B, Nq, Hq, Hkv, d = (case[x] for x in ("B", "Nq", "Hq", "Hkv", "d"))
    G, vec = Hq // Hkv, _mask_vectors(case)
    o = torch.zeros(B, Nq, Hq, d, dtype=F64, device="cuda")
    lse = torch.full((B, Hq, Nq), -math.inf, dtype=F64, device="cuda")
    for b, L in enumerate(s["lens_host"].tolist()):
        k, v = _sequence(s, "k", b, L), _sequence(s, "v", b, L)
        q = s["q"][b].double()
        j = torch.arange(L, device="cuda")
        for i in range(Nq):
            p = L - Nq + i
            hide = (j > p)[None]
            if vec is not None:
                a, e, f, g = (torch.from_numpy(x[b, :, :L]).cuda() for x in vec)
                hide = hide | ((a <= p) & (p < e)) | ((f <= p) & (p < g))
            x = torch.einsum("ghd,jhd->hgj", q[i].view(Hkv, G, d).transpose(0, 1), k).reshape(Hq, L) * d ** -0.5
            x = x.masked_fill(hide, -math.inf)
            z = torch.logsumexp(x, -1)
            w = torch.exp(x - z[:, None]).nan_to_num(0.0)
            o[b, i] = torch.einsum("hgj,jhd->hgd", w.view(Hkv, G, L), v).reshape(Hq, d)
            lse[b, :, i] = z
    return o, lse


def exact(case, seed):
    if case["op"] == "attention" and case["B"] * case["Nq"] > 2000:
        return None
    s = prepare(case, seed)
    if case["op"] == "attention":
        return _exact_attention(s)
    return _exact_gather(s, case["hi"]) if case["op"] == "gather" else _exact_append(s)
