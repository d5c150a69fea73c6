"""The cases that the norm and adapter operators are measured on.

Two operators of the block around a quantized projection:

* ``norm``: ``qlinear_block_norm``. The norm before a block with its AdaLN modulation
  (h from the residual stream), the norm after a block with its gate and the
  scaled residual (the next residual stream), or both in one pass between two blocks.
* ``adapters``: ``qlinear_adapters``. Low-rank adapters of many requests added
  to a projection that they share, plain or with the SwiGLU or gated-residual epilogue.

``own = False`` computes the plain form in elementary torch operations;
``own = True`` calls the library. ``exact`` is the definition in 64 bits.
"""
import random

import torch

own = False

DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
SIZES = {"f32": 4, "bf16": 2, "f16": 2}


# ------------------------------------------------------------------ cases

def _norm(name, M, D, kind, parts, y, residual, samples, ragged=False, affine=False, shift=False, residual_scale=1.0):
    """parts: "before", "after" or "between". ragged: rows mapped to samples by an index, the last rows to none."""
    return {"name": name, "op": "norm", "M": M, "D": D, "kind": kind, "parts": parts, "y": y, "residual": residual,
            "samples": samples, "ragged": ragged, "affine": affine, "shift": shift, "residual_scale": residual_scale}


def _adapters(name, M, K, N, rank, adapters, used, requests, base, y, out, table="bf16", epilogue="none", odd_ranks=False):
    """used: adapters that occur among the requests; base: whether the last request runs without one."""
    return {"name": name, "op": "adapters", "M": M, "K": K, "N": N, "rank": rank, "adapters": adapters, "used": used,
            "requests": requests, "base": base, "y": y, "out": out, "table": table, "epilogue": epilogue, "odd_ranks": odd_ranks}


def listed():
    return [
        # one conditioning token: the norm before its projection, where the launch is what counts
        _norm("before_1_row", 1, 4608, "rms", "before", None, "bf16", 1),
        # the 4096 image tokens of a 1024^2 image before QKV: RMS norm and AdaLN scale, bf16 stream
        _norm("before_image", 4096, 4608, "rms", "before", None, "bf16", 1),
        # after attention-out: fp32 product of the GEMM, RMS norm with weight, gate, fp32 stream
        _norm("after_image_f32", 4096, 4608, "rms", "after", "f32", "f32", 1, affine=True),
        # a packed batch of requests of unequal lengths, padded at its end, an odd width, LayerNorm with shift on both sides
        _norm("between_ragged_odd", 1001, 1003, "layer", "between", "f32", "bf16", 5, ragged=True, affine=True, shift=True),
        # four 2048^2 images between two blocks, everything in one pass: the largest stream
        _norm("between_images", 16896, 4608, "rms", "between", "bf16", "bf16", 4, affine=True, residual_scale=0.5),
        # the concatenated text-encoder features before the conditioning projection: very wide rows, LayerNorm
        _norm("before_text_wide", 512, 53248, "layer", "before", None, "bf16", 1, affine=True),
        # AdaLN modulation of one sample: one row, a wide output
        _adapters("one_row", 1, 4608, 27648, 16, 8, 1, 1, False, "f32", "f32"),
        # sixteen requests of one row, each with an adapter of its own
        _adapters("rows_16_distinct", 16, 4608, 4608, 16, 32, 16, 16, False, "f32", "f32"),
        # an odd batch of short requests, odd ranks below the table's, odd width, fp16 tables, some rows without an adapter
        _adapters("mixed_odd", 203, 512, 1003, 40, 12, 9, 14, True, "bf16", "bf16", table="f16", odd_ranks=True),
        # QKV of 4608 tokens of three requests
        _adapters("qkv", 4608, 4608, 13824, 32, 8, 3, 3, False, "f32", "f32"),
        # gate/up projection of two requests with the SwiGLU in the same pass
        _adapters("gate_up_swiglu", 4096, 4608, 24576, 16, 8, 2, 2, False, "bf16", "bf16", epilogue="swiglu"),
        # down projection of four 2048^2 requests, one without an adapter, with the gated residual update
        _adapters("down_gated", 16896, 12288, 4608, 64, 8, 3, 4, True, "bf16", "bf16", epilogue="gate"),
    ]


def _log_int(rng, lo, hi):
    return int(round(lo * (hi / lo) ** rng.random()))


def draw(rng):
    if rng.random() < 0.5:
        D = _log_int(rng, 64, 53248)
        if rng.random() < 0.6:
            D = max(64, D // 64 * 64)
        M = _log_int(rng, 1, max(1, min(16896, 16896 * 4608 // D)))
        parts = rng.choice(["before", "after", "between"])
        y = None if parts == "before" else rng.choice(["f32", "bf16"])
        residual = rng.choice(["f32", "bf16"])
        if parts == "between" and y == "f32" or residual == "f32":
            M = max(1, M // 2)
        case = _norm("", M, D, rng.choice(["rms", "layer"]), parts, y, residual, rng.randint(1, min(8, M)),
                     ragged=rng.random() < 0.5, affine=rng.random() < 0.5, shift=rng.random() < 0.5,
                     residual_scale=rng.choice([1.0, 0.5]))
        del case["name"]
        return case
    K = 64 * _log_int(rng, 2, 192)
    epilogue = rng.choice(["none", "none", "swiglu", "gate"])
    N = _log_int(rng, 64, 27648)
    if epilogue == "swiglu":
        N = N // 2 * 2
    # the largest listed case moves 16896 * (12288 + 3 * 4608) halves
    M = _log_int(rng, 1, max(1, min(16896, 16896 * 12288 // (K + 6 * N))))
    rank = 8 * _log_int(rng, 1, 16)
    adapters = _log_int(rng, 1, 32)
    requests = rng.randint(1, min(M, 32))
    base = requests > 1 and rng.random() < 0.5
    used = rng.randint(1, max(1, min(adapters, requests - int(base))))
    case = _adapters("", M, K, N, rank, adapters, used, requests, base, rng.choice(["f32", "bf16"]),
                     rng.choice(["f32", "bf16"]), table=rng.choice(["bf16", "bf16", "f16"]), epilogue=epilogue,
                     odd_ranks=rng.random() < 0.5)
    del case["name"]
    return case


def _lengths(M, parts, key):
    """M rows as `parts` runs of unequal lengths, the same for every seed."""
    r = random.Random(1000003 * M + 101 * parts + key)
    cuts = sorted(r.sample(range(1, M), parts - 1)) if parts > 1 else []
    edges = [0] + cuts + [M]
    return [b - a for a, b in zip(edges, edges[1:])]


def _pad_rows(case):
    """Rows behind the last sample of a ragged batch."""
    return case["M"] // 16 if case["ragged"] else 0


def _slot_ranks(case):
    """Effective ranks of the adapters in use, in the order the requests take them."""
    r = random.Random(case["rank"] * 7 + case["used"])
    return [r.randint(1, case["rank"]) if case["odd_ranks"] else case["rank"] for _ in range(case["used"])]


def _request_slots(case):
    """Per request the slot (0 .. used - 1) of its adapter, None for the request without one."""
    n = case["requests"] - int(case["base"])
    return [i % case["used"] for i in range(n)] + [None] * int(case["base"])


# ------------------------------------------------------------------ inputs

def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _prepare_norm(case, seed):
    g = _gen(seed)
    M, D, S = case["M"], case["D"], case["samples"]
    normal = lambda *shape: torch.randn(shape, generator=g, device="cuda")  # noqa: E731
    st = {"case": case}
    # a residual stream grows over the blocks and has a few large channels; a block's output is nearer to one
    channels = 1.0 + 8.0 * (torch.rand(D, generator=g, device="cuda") < 0.01)
    st["residual"] = (normal(M, D) * channels * 2.0 + 0.1).to(DTYPES[case["residual"]])
    before, after = case["parts"] != "after", case["parts"] != "before"
    # one modulation output per sample, its pieces taken as views (shift, scale, gate)
    mod = torch.empty((S, 3, D), device="cuda")
    mod[:, 0] = 0.2 * normal(S, D)
    mod[:, 1] = 0.3 * normal(S, D)
    mod[:, 2] = torch.tanh(normal(S, D))
    st["scale"] = mod[:, 1] if before else None
    st["shift"] = mod[:, 0] if before and case["shift"] else None
    st["gate"] = mod[:, 2] if after else None
    if after:
        st["y"] = (normal(M, D) * 0.7).to(DTYPES[case["y"]])
    weight = lambda: 1.0 + 0.2 * normal(D)  # noqa: E731
    st["w_post"] = weight() if after and case["affine"] else None
    st["w_pre"] = weight() if before and case["affine"] else None
    if case["ragged"]:
        pad = _pad_rows(case)
        rows = torch.tensor(_lengths(M - pad, S, 1) + [pad]) if pad else torch.tensor(_lengths(M, S, 1))
        ids = torch.tensor(list(range(S)) + ([-1] if pad else []))
        st["row_sample"] = torch.repeat_interleave(ids, rows).to(torch.int32).cuda()
        st["mod_rows"] = 0
    else:
        st["row_sample"] = None
        st["mod_rows"] = -(-M // S)
    # the buffers that the step writes: what lies behind the last sample has to stay
    st["residual_out"] = torch.zeros((M, D), dtype=DTYPES[case["residual"]], device="cuda") if after else None
    st["h"] = torch.zeros((M, D), dtype=torch.bfloat16, device="cuda") if before else None
    return st


def _prepare_adapters(case, seed):
    g = _gen(seed)
    M, K, N, R, n = case["M"], case["K"], case["N"], case["rank"], case["adapters"]
    normal = lambda *shape: torch.randn(shape, generator=g, device="cuda")  # noqa: E731
    table = DTYPES[case["table"]]
    st = {"case": case}
    st["x"] = normal(M, K).to(torch.bfloat16)
    st["a"] = (normal(n, R, K) / K ** 0.5).to(table)
    st["b"] = (normal(n, N, R) * (0.5 / R ** 0.5)).to(table)
    st["y"] = normal(M, N).to(DTYPES[case["y"]])
    order = random.Random(seed).sample(range(n), case["used"])
    ids = torch.tensor([-1 if s is None else order[s] for s in _request_slots(case)])
    rows = torch.tensor(_lengths(M, case["requests"], 2))
    st["row_adapter"] = torch.repeat_interleave(ids, rows).to(torch.int32).cuda()
    ranks = [R] * n
    for slot, r in enumerate(_slot_ranks(case)):
        ranks[order[slot]] = r
    st["ranks"] = torch.tensor(ranks, dtype=torch.int32, device="cuda") if case["odd_ranks"] else None
    st["scaling"] = 0.5 + torch.rand(n, generator=g, device="cuda")
    st["mod_rows"] = -(-M // 4)
    if case["epilogue"] == "gate":
        st["residual"] = normal(M, N).to(DTYPES[case["out"]])
        st["gate"] = torch.tanh(normal(-(-M // st["mod_rows"]), N))
    return st


def prepare(case, seed):
    return _prepare_norm(case, seed) if case["op"] == "norm" else _prepare_adapters(case, seed)


# ------------------------------------------------------------------ one pass

EPS = 1e-6


def _normalise(v, kind):
    if kind == "layer":
        v = v - v.mean(dim=1, keepdim=True)
    return v * torch.rsqrt((v * v).mean(dim=1, keepdim=True) + EPS)


def _plain_norm(st):
    case = st["case"]
    M = case["M"]
    if st["row_sample"] is not None:
        sample = st["row_sample"].long()
        live = (sample >= 0)[:, None]
        sample = sample.clamp(min=0)
    else:
        sample, live = torch.arange(M, device="cuda") // st["mod_rows"], None
    out = {}
    r = case["residual_scale"] * st["residual"].float()
    if case["parts"] != "before":
        z = _normalise(st["y"].float(), case["kind"])
        if st["w_post"] is not None:
            z = z * st["w_post"]
        r = r + st["gate"][sample] * z
        new = r.to(st["residual_out"].dtype)
        out["residual"] = new if live is None else torch.where(live, new, st["residual_out"])
    if case["parts"] != "after":
        h = _normalise(r, case["kind"])
        if st["w_pre"] is not None:
            h = h * st["w_pre"]
        h = h * (1.0 + st["scale"][sample])
        if st["shift"] is not None:
            h = h + st["shift"][sample]
        new = h.to(torch.bfloat16)
        out["h"] = new if live is None else torch.where(live, new, st["h"])
    return out


def _plain_adapters(st):
    case = st["case"]
    n, R, K = st["a"].shape
    # every row against every adapter of the table, then each row keeps its own adapter's columns
    v = st["x"].float() @ st["a"].float().reshape(n * R, K).T
    column = torch.arange(n * R, device="cuda")
    keep = st["row_adapter"][:, None] == (column // R)[None]
    if st["ranks"] is not None:
        keep = keep & (column % R < st["ranks"][column // R])[None]
    v = torch.where(keep, v * st["scaling"][column // R], 0.0)
    t = st["y"].float() + v @ st["b"].float().transpose(1, 2).reshape(n * R, -1)
    if case["epilogue"] == "swiglu":
        F = t.shape[1] // 2
        t = t[:, :F] / (1.0 + torch.exp(-t[:, :F])) * t[:, F:]
    elif case["epilogue"] == "gate":
        rows = torch.arange(t.shape[0], device="cuda") // st["mod_rows"]
        t = st["residual"].float() + st["gate"][rows] * t
    return t.to(DTYPES[case["out"]])


def _own_norm(st):
    from group_wise_affine_qlinear_amd import qlinear as ql
    case = st["case"]
    kind = ql.QL_NORM_RMS if case["kind"] == "rms" else ql.QL_NORM_LAYER
    before, after = case["parts"] != "after", case["parts"] != "before"
    ql.qlinear_block_norm(
        st["residual"], case["M"], case["D"], y=st.get("y"), residual_scale=case["residual_scale"],
        post_norm=kind if after else ql.QL_NORM_NONE, post_weight=st["w_post"], post_eps=EPS, gate=st["gate"],
        residual_out=st["residual_out"],
        pre_norm=kind if before else ql.QL_NORM_NONE, pre_weight=st["w_pre"], pre_eps=EPS, scale=st["scale"],
        shift=st["shift"], h=st["h"], mod_rows=st["mod_rows"], row_sample=st["row_sample"])
    out = {}
    if after:
        out["residual"] = st["residual_out"]
    if before:
        out["h"] = st["h"]
    return out


def _own_adapters(st):
    from group_wise_affine_qlinear_amd import qlinear as ql
    case = st["case"]
    M, K, N = case["M"], case["K"], case["N"]
    more = {}
    if case["epilogue"] == "swiglu":
        more = {"epilogue": ql.QL_EPI_SWIGLU}
    elif case["epilogue"] == "gate":
        more = {"epilogue": ql.QL_EPI_GATE_RESIDUAL, "residual": st["residual"], "gate": st["gate"],
                "gate_rows": st["mod_rows"]}
    out = torch.empty((M, N // 2 if case["epilogue"] == "swiglu" else N), dtype=DTYPES[case["out"]], device="cuda")
    return ql.qlinear_adapters(st["x"], st["a"], st["b"], st["row_adapter"], M, N, K, out, y=st["y"], ranks=st["ranks"],
                               scaling=st["scaling"], **more)


def run(state):
    if own:
        return _own_norm(state) if state["case"]["op"] == "norm" else _own_adapters(state)
    return _plain_norm(state) if state["case"]["op"] == "norm" else _plain_adapters(state)


# ------------------------------------------------------------------ the least work, and the definition

def work(case):
    if case["op"] == "norm":
        before, after = case["parts"] != "after", case["parts"] != "before"
        rows, D = case["M"] - _pad_rows(case), case["D"]
        per = SIZES[case["residual"]] * (2 if after else 1) + (SIZES[case["y"]] if after else 0) + (2 if before else 0)
        vectors = case["samples"] * (int(after) + int(before) * (1 + int(case["shift"])))
        vectors += int(case["affine"]) * (int(after) + int(before))
        flops = rows * D * (8 * int(after) + 8 * int(before))
        return {"bytes": rows * D * per + 4 * D * vectors + (4 * case["M"] if case["ragged"] else 0), "flops": flops}
    M, K, N = case["M"], case["K"], case["N"]
    lengths, slots, ranks = _lengths(M, case["requests"], 2), _request_slots(case), _slot_ranks(case)
    rows = sum(n for n, s in zip(lengths, slots) if s is not None)
    products = sum(n * ranks[s] for n, s in zip(lengths, slots) if s is not None)
    width = N // 2 if case["epilogue"] == "swiglu" else N
    total = rows * K * 2 + sum(ranks) * (K + N) * 2 + M * N * SIZES[case["y"]] + M * width * SIZES[case["out"]] + 4 * M
    if case["epilogue"] == "gate":
        total += M * N * SIZES[case["out"]] + min(4, M) * N * 4
    return {"bytes": total, "flops": 2 * products * (K + N) + M * N}


def _exact_norm(st):
    case = st["case"]
    D, f64 = case["D"], torch.float64

    def unit(v):
        if case["kind"] == "layer":
            v = v - v.sum(dim=1, keepdim=True) / D
        return v / torch.sqrt((v ** 2).sum(dim=1, keepdim=True) / D + EPS)

    outs = {"residual": st["residual_out"], "h": st["h"]}
    outs = {k: torch.zeros(v.shape, dtype=f64, device="cuda") for k, v in outs.items() if v is not None}
    owner = st["row_sample"].tolist() if st["row_sample"] is not None else [m // st["mod_rows"] for m in range(case["M"])]
    for s in range(case["samples"]):
        rows = [m for m, o in enumerate(owner) if o == s]
        if not rows:
            continue
        part = slice(rows[0], rows[-1] + 1)
        r = st["residual"][part].to(f64) * case["residual_scale"]
        if case["parts"] != "before":
            z = unit(st["y"][part].to(f64))
            if st["w_post"] is not None:
                z = z * st["w_post"].to(f64)
            r = r + st["gate"][s].to(f64) * z
            outs["residual"][part] = r
        if case["parts"] != "after":
            h = unit(r)
            if st["w_pre"] is not None:
                h = h * st["w_pre"].to(f64)
            h = h + h * st["scale"][s].to(f64)
            if st["shift"] is not None:
                h = h + st["shift"][s].to(f64)
            outs["h"][part] = h
    return outs


def _exact_adapters(st):
    case = st["case"]
    f64 = torch.float64
    t = st["y"].to(f64)
    owner = st["row_adapter"].tolist()
    for a in sorted(set(o for o in owner if o >= 0)):
        rows = torch.tensor([m for m, o in enumerate(owner) if o == a], device="cuda")
        r = case["rank"] if st["ranks"] is None else int(st["ranks"][a])
        v = torch.mm(st["x"][rows].to(f64), st["a"][a, :r].to(f64).T.contiguous())
        t[rows] += float(st["scaling"][a]) * torch.mm(v, st["b"][a, :, :r].to(f64).T.contiguous())
    if case["epilogue"] == "swiglu":
        g, u = t.chunk(2, dim=1)
        return g * torch.sigmoid(g) * u
    if case["epilogue"] == "gate":
        for m0 in range(0, case["M"], st["mod_rows"]):
            part = slice(m0, min(case["M"], m0 + st["mod_rows"]))
            t[part] = t[part] * st["gate"][m0 // st["mod_rows"]].to(f64) + st["residual"][part].to(f64)
    return t


def exact(case, seed):
    st = prepare(case, seed)
    return _exact_norm(st) if case["op"] == "norm" else _exact_adapters(st)
