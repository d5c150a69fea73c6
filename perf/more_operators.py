"""The cases that the operators between a QKV projection and the output projection are measured on.

* ``rope``: ``qlinear_qk_norm_rope``. What a fused projection wrote becomes the heads that attention reads: each
  query and key head is normalised and rotated by its positions on one or more axes (time, height, width), the
  values are rounded, all in one pass.
* ``attention``: ``qlinear_attention``. Packed samples of queries over their own keys, as many as the queries or
  another length (an encoder's states), with shared key heads and masked keys, down to single queries.

``own = False`` computes the plain form in elementary torch operations;
``own = True`` calls the library. ``exact`` is the definition in 64 bits.
"""
import random

import torch

own = False

DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16}
SIZES = {"f32": 4, "bf16": 2}


# ------------------------------------------------------------------ cases

def _rope(name, M, q_heads, kv_heads, D, source, norm="rms", layout="halves", rotary=None, axes=3, order="own", far=0,
          pad=False):
    """source: type of the projection's output. rotary: dimensions that turn. far: the first position. pad: rows behind the last sample."""
    return {"name": name, "op": "rope", "M": M, "q_heads": q_heads, "kv_heads": kv_heads, "D": D, "source": source,
            "norm": norm, "layout": layout, "rotary": D if rotary is None else rotary, "axes": axes, "order": order,
            "far": far, "pad": pad}


def _attention(name, queries, keys, q_heads, kv_heads, D, samples=1, masked=False, packed=False):
    """masked: a mask over the keys, one sample without any. packed: q, k and v as slices of one buffer."""
    return {"name": name, "op": "attention", "queries": queries, "keys": keys, "q_heads": q_heads, "kv_heads": kv_heads,
            "D": D, "samples": samples, "masked": masked, "packed": packed}


def listed():
    return [
        # one token of one request: the launch is what counts
        _rope("rope_1_row", 1, 18, 18, 256, "f32", axes=1),
        # text tokens far into a long context, shared key heads, sections of one frequency table
        _rope("rope_text_far", 2047, 32, 8, 128, "bf16", order="shared", far=100000),
        # a packed odd batch, padded at its end: LayerNorm, neighbouring pairs, part of the head turned, two axes
        _rope("rope_odd_padded", 1001, 24, 8, 72, "bf16", norm="layer", layout="pairs", rotary=40, axes=2, pad=True),
        # the 4096 image and 512 text tokens of a 1024^2 image, fp32 output of the QKV projection
        _rope("rope_image", 4608, 18, 18, 256, "f32"),
        # four 2048^2 images: the largest streams
        _rope("rope_images", 16896, 18, 18, 256, "f32", order="turns"),
        # one query over the text states of its request
        _attention("one_query", 1, 512, 18, 18, 256),
        # sixteen requests of one query each over caches of unequal lengths, shared key heads
        _attention("queries_16", 16, 65536, 32, 8, 128, samples=16),
        # a packed odd batch over padded encoder states, an odd head, one request whose states are all masked
        _attention("cross_odd_masked", 1171, 731, 16, 16, 72, samples=5, masked=True),
        # image tokens over the text states
        _attention("cross_text", 4096, 512, 18, 18, 256),
        # a few learned queries over the states of a large image
        _attention("few_over_many", 77, 16896, 24, 24, 128),
        # the tokens of one 1024^2 image and its text among themselves, read from the buffer that the pass before wrote
        _attention("image", 4608, 4608, 18, 18, 256, packed=True),
        # a 2048^2 image and its text among themselves: the largest
        _attention("image_large", 16896, 16896, 18, 18, 256, packed=True),
    ]


def _log_int(rng, lo, hi):
    return int(round(lo * (hi / lo) ** rng.random()))


def draw(rng):
    D = 8 * rng.choice([4, 8, 8, 9, 10, 12, 14, 16, 16, 16, 20, 24, 28, 32, 32, 32])
    kv_heads = rng.choice([1, 2, 4, 8, 12, 18])
    q_heads = kv_heads * rng.choice([1, 1, 1, 2, 3, 4, 8])
    if rng.random() < 0.4:
        source = rng.choice(["f32", "bf16"])
        # the largest listed case holds 16896 rows of 54 heads of 256
        M = _log_int(rng, 1, max(1, min(16896, 16896 * 54 * 256 // ((q_heads + 2 * kv_heads) * D))))
        rotary = D if rng.random() < 0.7 else 8 * rng.randint(1, D // 8)
        case = _rope("", M, q_heads, kv_heads, D, source, norm=rng.choice(["none", "rms", "rms", "layer"]),
                     layout=rng.choice(["halves", "pairs"]), rotary=rotary, axes=rng.randint(1, min(3, rotary // 2)),
                     order=rng.choice(["own", "shared", "turns"]), far=rng.choice([0, 0, 1000, 1000000]),
                     pad=M > 16 and rng.random() < 0.3)
    else:
        queries = _log_int(rng, 1, 16896)
        keys = queries if rng.random() < 0.3 else _log_int(rng, 1, 65536)
        # no more products than the largest listed case, and no more scores for the plain form, of all heads and of a key head's
        most = 16896 * 16896 * 18 * 256 // (q_heads * max(D, 256))
        most = min(most, 16896 * 16896 * kv_heads // q_heads)
        if queries * keys > most:
            keys = max(1, most // queries)
        samples = rng.randint(1, min(8, queries, keys))
        case = _attention("", queries, keys, q_heads, kv_heads, D, samples=samples, masked=rng.random() < 0.3,
                          packed=queries == keys and rng.random() < 0.5)
    del case["name"]
    return case


def _lengths(total, parts, key):
    """`total` rows as `parts` runs of unequal lengths, the same for every seed."""
    r = random.Random(1000003 * total + 101 * parts + key)
    cuts = sorted(r.sample(range(1, total), parts - 1)) if parts > 1 else []
    edges = [0] + cuts + [total]
    return [b - a for a, b in zip(edges, edges[1:])]


def _pad_rows(case):
    return case["M"] // 16 if case["pad"] else 0


def _key_lengths(case):
    """Keys of each sample; packed q, k and v have the samples of the queries."""
    return _lengths(case["keys"], case["samples"], 1 if case["queries"] == case["keys"] else 2)


def _kept_keys(case):
    """Unmasked keys of each sample: a prefix of its states. The last of several samples has none."""
    lengths = _key_lengths(case)
    if not case["masked"]:
        return lengths
    kept = [max(1, n - n // (4 + i)) for i, n in enumerate(lengths)]
    if len(kept) > 1:
        kept[-1] = 0
    return kept


# ------------------------------------------------------------------ inputs

def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


THETA = 10000.0


def _sections(case):
    """Pairs of each axis."""
    pairs, axes = case["rotary"] // 2, case["axes"]
    each = pairs // axes
    return [pairs - each * (axes - 1)] + [each] * (axes - 1)


def _table(case):
    """(frequency, axis) of each pair. own: every axis has the frequencies of its own pairs; shared: those of all
    pairs, in runs; turns: those of all pairs, the axes in turn while they have pairs left."""
    sections, pairs = _sections(case), case["rotary"] // 2
    if case["order"] == "own":
        return [(THETA ** (-j / n), a) for a, n in enumerate(sections) for j in range(n)]
    if case["order"] == "shared":
        axis = [a for a, n in enumerate(sections) for _ in range(n)]
    else:
        axis = [a for turn in range(max(sections)) for a, n in enumerate(sections) if turn < n]
    return [(THETA ** (-i / pairs), a) for i, a in enumerate(axis)]


def _prepare_rope(case, seed):
    g = _gen(seed)
    M, D, hq, hkv = case["M"], case["D"], case["q_heads"], case["kv_heads"]
    # a projection's output: some channels are larger than the rest
    channels = 1.0 + 4.0 * (torch.rand(hq + 2 * hkv, D, generator=g, device="cuda") < 0.02)
    qkv = (torch.randn(M, hq + 2 * hkv, D, generator=g, device="cuda") * channels + 0.05).to(DTYPES[case["source"]])
    st = {"case": case, "qkv": qkv}
    st["q"], st["k"], st["v"] = qkv[:, :hq], qkv[:, hq:hq + hkv], qkv[:, hq + hkv:]
    weight = lambda: 1.0 + 0.2 * torch.randn(D, generator=g, device="cuda")  # noqa: E731
    st["q_weight"], st["k_weight"] = (None, None) if case["norm"] == "none" else (weight(), weight())
    table = _table(case)
    st["freqs"] = torch.tensor([f for f, _ in table], dtype=torch.float32, device="cuda")
    st["pair_axis"] = torch.tensor([a for _, a in table], dtype=torch.int32, device="cuda")
    # text first, the same number on every axis, then an image in rows
    first, text = case["far"] + int(torch.randint(0, 100, (1,), generator=g, device="cuda")), max(1, M // 9)
    i = torch.arange(M, device="cuda")
    width = max(1, int((M - text) ** 0.5))
    at = (i - text).clamp(min=0)
    image = [torch.full_like(i, text), text + at // width, text + at % width]
    st["positions"] = torch.stack([first + torch.where(i < text, i, image[a]) for a in range(case["axes"])]).to(torch.int32)
    st["rows_end"] = torch.tensor([M - _pad_rows(case)], dtype=torch.int32, device="cuda") if case["pad"] else None
    # the buffers that the step writes: what lies behind the last sample has to stay
    new = lambda heads: torch.zeros((M, heads, D), dtype=torch.bfloat16, device="cuda")  # noqa: E731
    st["q_out"], st["k_out"], st["v_out"] = new(hq), new(hkv), new(hkv)
    return st


def _prepare_attention(case, seed):
    g = _gen(seed)
    D, hq, hkv, S = case["D"], case["q_heads"], case["kv_heads"], case["samples"]
    nq, nk = case["queries"], case["keys"]
    st = {"case": case}
    if case["packed"]:
        qkv = torch.empty((nq, hq + 2 * hkv, D), dtype=torch.bfloat16, device="cuda")
        st["q"], st["k"], st["v"] = qkv[:, :hq], qkv[:, hq:hq + hkv], qkv[:, hq + hkv:]
    else:
        new = lambda n, heads: torch.empty((n, heads, D), dtype=torch.bfloat16, device="cuda")  # noqa: E731
        st["q"], st["k"], st["v"] = new(nq, hq), new(nk, hkv), new(nk, hkv)
    normal = lambda t: torch.randn(t.shape, generator=g, device="cuda")  # noqa: E731
    # normalised heads: scores of a spread of about two; values have a mean of their own in every channel
    st["q"].copy_(normal(st["q"]) * 2.0)
    st["k"].copy_(normal(st["k"]) + 0.5 * torch.randn(1, hkv, D, generator=g, device="cuda"))
    st["v"].copy_(normal(st["v"]) + 0.5 * torch.randn(1, hkv, D, generator=g, device="cuda"))
    st["key_mask"] = None
    if case["masked"]:
        keep = torch.tensor([b for n, kept in zip(_key_lengths(case), _kept_keys(case)) for b in [True] * kept + [False] * (n - kept)])
        st["key_mask"] = keep.cuda()
        # what nobody wrote
        st["k"][~st["key_mask"]] = float("nan")
        st["v"][~st["key_mask"]] = float("nan")
    edges = lambda lengths: torch.tensor([0] + lengths, dtype=torch.int32).cumsum(0).to(torch.int32).cuda()  # noqa: E731
    st["q_offsets"] = edges(_lengths(nq, S, 1)) if S > 1 else None
    st["k_offsets"] = edges(_key_lengths(case)) if S > 1 else None
    st["out"] = torch.zeros((nq, hq, D), dtype=torch.bfloat16, device="cuda")
    return st


def prepare(case, seed):
    return _prepare_rope(case, seed) if case["op"] == "rope" else _prepare_attention(case, seed)


# ------------------------------------------------------------------ one pass

EPS = 1e-6


def _plain_turn(st, x, weight):
    """Norm and rotation of [M, heads, D]."""
    case = st["case"]
    x = x.float()
    if case["norm"] == "layer":
        x = x - x.mean(dim=-1, keepdim=True)
    if case["norm"] != "none":
        x = x * torch.rsqrt((x * x).mean(dim=-1, keepdim=True) + EPS) * weight
    R = case["rotary"]
    angle = st["positions"][st["pair_axis"].long()].double() * st["freqs"].double()[:, None]  # [pairs, M]
    cos, sin = angle.cos().float().T[:, None], angle.sin().float().T[:, None]
    if case["layout"] == "halves":
        a, b = x[..., :R // 2], x[..., R // 2:R]
        turned = torch.cat([a * cos - b * sin, b * cos + a * sin], dim=-1)
    else:
        a, b = x[..., 0:R:2], x[..., 1:R:2]
        turned = torch.stack([a * cos - b * sin, b * cos + a * sin], dim=-1).flatten(-2)
    return torch.cat([turned, x[..., R:]], dim=-1).to(torch.bfloat16)


def _plain_rope(st):
    out = {"q": _plain_turn(st, st["q"], st["q_weight"]), "k": _plain_turn(st, st["k"], st["k_weight"]),
           "v": st["v"].to(torch.bfloat16)}
    if st["rows_end"] is not None:
        live = (torch.arange(st["case"]["M"], device="cuda") < st["rows_end"])[:, None, None]
        out = {n: torch.where(live, t, st[n + "_out"]) for n, t in out.items()}
    return out


def _plain_attention(st):
    case = st["case"]
    nq, nk, D, hkv = case["queries"], case["keys"], case["D"], case["kv_heads"]
    group = case["q_heads"] // hkv
    keep = None
    if st["q_offsets"] is not None:
        # the sample of each query and each key
        sq = torch.searchsorted(st["q_offsets"], torch.arange(nq, device="cuda", dtype=torch.int32), right=True)
        sk = torch.searchsorted(st["k_offsets"], torch.arange(nk, device="cuda", dtype=torch.int32), right=True)
        keep = (sq[:, None] == sk[None]).repeat(group, 1)
    k, v = st["k"].float(), st["v"].float()
    if st["key_mask"] is not None:
        k = torch.where(st["key_mask"][:, None, None], k, 0.0)
        v = torch.where(st["key_mask"][:, None, None], v, 0.0)
        keep = st["key_mask"][None] if keep is None else keep & st["key_mask"][None]
    # [kv_heads, group * queries, D] against the keys that the group shares
    q = st["q"].float().reshape(nq, hkv, group, D).permute(1, 2, 0, 3).reshape(hkv, group * nq, D)
    s = torch.bmm(q, k.permute(1, 2, 0).contiguous()).mul_(D ** -0.5)
    if keep is not None:
        s.masked_fill_(~keep[None], float("-inf"))
    s = s.sub_(s.amax(dim=-1, keepdim=True).clamp_(min=-1e30)).exp_()
    total = s.sum(dim=-1, keepdim=True)
    o = torch.bmm(s, v.permute(1, 0, 2).contiguous()) / torch.where(total > 0, total, 1.0)
    return o.reshape(hkv, group, nq, D).permute(2, 0, 1, 3).reshape(nq, hkv * group, D).to(torch.bfloat16)


def _own_rope(st):
    from group_wise_affine_qlinear_amd import qlinear as ql
    case = st["case"]
    norm = {"none": ql.QL_NORM_NONE, "rms": ql.QL_NORM_RMS, "layer": ql.QL_NORM_LAYER}[case["norm"]]
    layout = ql.QL_ROPE_HALVES if case["layout"] == "halves" else ql.QL_ROPE_PAIRS
    ql.qlinear_qk_norm_rope(case["M"], case["D"], q=st["q"], k=st["k"], v=st["v"], q_out=st["q_out"], k_out=st["k_out"],
                            v_out=st["v_out"], norm=norm, eps=EPS, q_weight=st["q_weight"], k_weight=st["k_weight"],
                            rope=layout, freqs=st["freqs"], pair_axis=st["pair_axis"], positions=st["positions"],
                            rows_end=st["rows_end"])
    return {"q": st["q_out"], "k": st["k_out"], "v": st["v_out"]}


def _own_attention(st):
    from group_wise_affine_qlinear_amd import qlinear as ql
    return ql.qlinear_attention(st["q"], st["k"], st["v"], st["out"], q_offsets=st["q_offsets"],
                                k_offsets=st["k_offsets"], key_mask=st["key_mask"])


def run(state):
    rope = state["case"]["op"] == "rope"
    if own:
        return _own_rope(state) if rope else _own_attention(state)
    return _plain_rope(state) if rope else _plain_attention(state)


# ------------------------------------------------------------------ the least work, and the definition

def work(case):
    D, hq, hkv = case["D"], case["q_heads"], case["kv_heads"]
    if case["op"] == "rope":
        rows, heads = case["M"] - _pad_rows(case), hq + 2 * hkv
        pairs = case["rotary"] // 2
        total = rows * (heads * D * (SIZES[case["source"]] + 2) + 4 * case["axes"]) + 8 * pairs
        if case["norm"] != "none":
            total += 8 * D
        flops = rows * (hq + hkv) * (6 * pairs + (0 if case["norm"] == "none" else 4 * D))
        return {"bytes": total, "flops": flops}
    kept = _kept_keys(case)
    products = sum(a * b for a, b in zip(_lengths(case["queries"], case["samples"], 1), kept))
    total = 2 * D * (2 * case["queries"] * hq + 2 * sum(kept) * hkv)
    if case["masked"]:
        total += case["keys"]
    return {"bytes": total, "flops": 4 * products * hq * D}


def _exact_rope(st):
    case, f64 = st["case"], torch.float64
    M, D, R = case["M"], case["D"], case["rotary"]
    rows = M - _pad_rows(case)
    unit = torch.ones(M, R // 2, dtype=torch.complex128, device="cuda")
    axis = st["pair_axis"].tolist()
    for i, f in enumerate(st["freqs"].tolist()):
        unit[:, i] = torch.polar(torch.ones(M, dtype=f64, device="cuda"), st["positions"][axis[i]].to(f64) * f)
    first = list(range(R // 2)) if case["layout"] == "halves" else list(range(0, R, 2))
    second = [i + R // 2 for i in first] if case["layout"] == "halves" else [i + 1 for i in first]
    out = {}
    for n in "qkv":
        x = st[n].to(f64)
        if n != "v":
            if case["norm"] == "layer":
                x = x - x.sum(dim=2, keepdim=True) / D
            if case["norm"] != "none":
                x = st[n + "_weight"].to(f64) * (x / torch.sqrt((x ** 2).sum(dim=2, keepdim=True) / D + EPS))
            z = torch.complex(x[:, :, first], x[:, :, second]) * unit[:, None]
            x = x.clone()
            x[:, :, first], x[:, :, second] = z.real, z.imag
        x[rows:] = 0.0
        out[n] = x
    return out


def _exact_attention(st):
    case, f64 = st["case"], torch.float64
    D, hq, hkv = case["D"], case["q_heads"], case["kv_heads"]
    out = torch.zeros(case["queries"], hq, D, dtype=f64, device="cuda")
    q0 = k0 = 0
    for nq, nk, kept in zip(_lengths(case["queries"], case["samples"], 1), _key_lengths(case), _kept_keys(case)):
        for h in range(hq if kept else 0):
            k = st["k"][k0:k0 + kept, h * hkv // hq].to(f64)
            v = st["v"][k0:k0 + kept, h * hkv // hq].to(f64).contiguous()
            for i in range(q0, q0 + nq, 8192):
                j = min(i + 8192, q0 + nq)
                s = torch.mm(st["q"][i:j, h].to(f64), k.T.contiguous()) / D ** 0.5
                out[i:j, h] = torch.mm(torch.softmax(s, dim=1), v)
        q0, k0 = q0 + nq, k0 + nk
    return out


def exact(case, seed):
    st = prepare(case, seed)
    return _exact_rope(st) if case["op"] == "rope" else _exact_attention(st)
