"""What differential attention and the rotation by several axes are measured on: cases, inputs,
plain forms and definitions.

  norm_rope_axes    per-head RMS norm and rotation of q and k where a token has a position on each
                    of several axes (time, height, width), each rotated pair going by one of them
  append_axes       the same for new tokens on their way into bf16 page pools; a token's slot goes
                    by its place in the context, its angles by its positions
  diff              differential attention, dense or packed: the difference of two softmax maps
                    over one set of values, with its per-head norm
  diff_chunk        the same for chunks of new tokens over a paged cache
  diff_decode       the same for one new token a sequence over a paged cache

A head of differential attention is d channels wide: two maps of d/2 channels side by side in
q and k, and one value row of d.
  A_m = softmax(scale q_m k_m^T),  y = A_1 v - lam A_2 v,
  O = out_scale * y * weight / sqrt(mean y^2 + eps)
"""
import math

import torch

own = False

# Hq, Hkv, d of this repository's configurations: the headline's grouped heads, the document
# workload's d = 64, and its decode's largest groups.
HEADS = {"gqa": (32, 8, 128), "mha64": (16, 16, 64), "wide": (64, 4, 64), "mqa": (12, 1, 128)}
EPS = 1e-5
OUT_SCALE = 0.8
GRID = (24, 16)  # patches of a frame, down and across


def listed():
    return [
        # four sequences' next tokens, q and k of two maps: the smallest call, one launch's latency
        {"name": "norm_rope_axes_step", "op": "norm_rope_axes", "heads": "gqa", "maps": 2,
         "batch": 4, "rows": 1, "far": 16384, "rot": 64, "axes": 3, "turns": False,
         "interleaved": False, "norm": True},
        # two prompts of 8192 tokens of video: runs of pairs for time, height and width
        {"name": "norm_rope_axes_video", "op": "norm_rope_axes", "heads": "gqa", "maps": 1,
         "batch": 2, "rows": 8192, "far": 8192, "rot": 128, "axes": 3, "turns": False,
         "interleaved": False, "norm": True},
        # one decode step of 32 sequences: 32 tokens scattered to 32 pages
        {"name": "append_axes_step", "op": "append_axes", "heads": "gqa", "maps": 2, "batch": 32,
         "lo": 256, "hi": 16384, "new": 1, "page": 64, "rot": 64, "axes": 3, "turns": False,
         "interleaved": False, "norm": True},
        # chunks of 16 prompts with images, small pages, the axes in turns
        {"name": "append_axes_chunks", "op": "append_axes", "heads": "gqa", "maps": 2,
         "batch": 16, "lo": 2048, "hi": 16384, "new": 2048, "page": 16, "rot": 64, "axes": 3,
         "turns": True, "interleaved": False, "norm": False},
        # a short prompt, no mask: few work units
        {"name": "diff_small", "op": "diff", "heads": "mha64", "batch": 1, "rows": 256,
         "mask": "none", "window": 0, "norm": True},
        # the headline prompt
        {"name": "diff_causal", "op": "diff", "heads": "gqa", "batch": 2, "rows": 8192,
         "mask": "causal", "window": 0, "norm": True},
        # a window over odd prompts, d = 64
        {"name": "diff_window", "op": "diff", "heads": "mha64", "batch": 3, "rows": 5003,
         "mask": "sliding", "window": 1000, "norm": True},
        # chunks of five odd prompts, 16 query heads a kv head, d = 64, small pages
        {"name": "diff_chunk_odd", "op": "diff_chunk", "heads": "wide", "batch": 5, "lo": 37,
         "hi": 1501, "new": 700, "page": 16, "norm": False},
        # 16 chunks of up to 2048 tokens over contexts of 2K to 16K
        {"name": "diff_chunk_batch", "op": "diff_chunk", "heads": "gqa", "batch": 16, "lo": 2048,
         "hi": 16384, "new": 2048, "page": 64, "norm": True},
        # one 16K-token sequence: the step's latency
        {"name": "diff_decode_one", "op": "diff_decode", "heads": "gqa", "batch": 1, "lo": 16384,
         "hi": 16384, "page": 64, "empty": 0, "norm": True},
        # the decode batch of the paged benchmark: 32 sequences of 1K to 16K tokens
        {"name": "diff_decode_batch", "op": "diff_decode", "heads": "gqa", "batch": 32, "lo": 1024,
         "hi": 16384, "page": 64, "empty": 0, "norm": True},
        # 16 query heads a kv head, d = 64, small pages, slots of a padded batch left empty
        {"name": "diff_decode_wide", "op": "diff_decode", "heads": "wide", "batch": 48, "lo": 1,
         "hi": 16384, "page": 16, "empty": 3, "norm": True},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    while True:  # nothing larger than the largest listed cases
        case = _draw(rng)
        w = work(case)
        if w["bytes"] < 1.1e9 and w["flops"] < 1.6e12:
            return case


def _draw(rng):
    op = rng.choice(["norm_rope_axes", "append_axes", "diff", "diff_chunk", "diff_decode"])
    heads = rng.choice(sorted(HEADS))
    case = {"op": op, "heads": heads}
    if op in ("norm_rope_axes", "append_axes"):
        maps = rng.choice([1, 2])
        row = HEADS[heads][2] // maps
        case.update(maps=maps, rot=rng.choice([16, row // 2, row, row]), axes=rng.choice([2, 3, 4]),
                    turns=rng.random() < 0.5, interleaved=rng.random() < 0.3,
                    norm=rng.random() < 0.6)
    if op == "norm_rope_axes":
        total = _log(rng, 1, 16000)
        batch = rng.choice([1, 2, 3, total])
        case.update(batch=batch, rows=max(1, total // batch), far=_log(rng, 64, 100000))
        return case
    if op == "diff":
        rows = _log(rng, 1, 8192)
        mask = rng.choice(["none", "causal", "causal", "sliding", "sliding_bidir", "prefix",
                           "document", "document_bidir"])
        case.update(batch=rng.choice([1, 2, 3, 5]), rows=rows, mask=mask,
                    window=_log(rng, 1, 4096), norm=rng.random() < 0.7)
        return case
    case.update(page=rng.choice([16, 32, 64, 128]))
    if op in ("append_axes", "diff_chunk"):
        hi = _log(rng, 8, 6000)
        new = 1 if rng.random() < 0.3 else _log(rng, 2, 2048)
        case.update(batch=_log(rng, 1, 16), lo=max(1, hi // rng.choice([1, 2, 8])), hi=hi, new=new)
        if op == "diff_chunk":
            case.update(norm=rng.random() < 0.7)
        return case
    hi = _log(rng, 2, 16384)
    case.update(batch=_log(rng, 1, 32), lo=max(1, hi // rng.choice([1, 4, 16])), hi=hi,
                empty=rng.choice([0, 0, 1, 2]), norm=rng.random() < 0.7)
    return case


# ------------------------------------------------------------------ shapes of a case

def _spread(n, lo, hi):
    """n whole numbers spread over lo .. hi in an order of their own: sizes go by the case alone,
    values by the seed."""
    step = (math.sqrt(5) - 1) / 2
    return [lo + int((hi - lo + 1) * ((0.5 + i * step) % 1.0)) for i in range(n)]


def _lengths(case):
    """(context lengths, new tokens) of the sequences."""
    lk = _spread(case["batch"], case["lo"], case["hi"])
    new = case["new"]
    if new <= 1:
        return lk, [new] * len(lk)
    step = math.sqrt(2) - 1
    lq = [max(1, int(min(new, L) * (0.125 + 0.875 * ((0.37 + i * step) % 1.0))))
          for i, L in enumerate(lk)]
    return lk, lq


def _decode_lengths(case):
    lk = _spread(case["batch"], case["lo"], case["hi"])
    for i in range(case["empty"]):
        if len(lk) > 1:
            lk[(7 * i + 1) % len(lk)] = 0
    return lk


def _segments(case):
    """Lengths of the packed segments of a document case: batch of them, of up to `rows`."""
    return _spread(case["batch"], max(1, case["rows"] // 16), case["rows"])


def _seen(case, n):
    """Visible (query, key) pairs of one head over a sequence of n tokens."""
    mask, w = case["mask"], case["window"]
    full, causal = n * n, n * (n + 1) // 2
    if mask in ("none", "document_bidir"):
        return full
    if mask in ("causal", "document"):
        return causal
    if mask == "sliding":
        w = min(w, n)
        return causal - (n - w) * (n - w + 1) // 2
    if mask == "sliding_bidir":
        out = max(0, n - 1 - w)
        return full - out * (out + 1)
    p = min(w, n)  # prefix
    return causal + p * (p - 1) // 2


def work(case):
    hq, hkv, d = HEADS[case["heads"]]
    row, op = 2 * d, case["op"]
    if op in ("norm_rope_axes", "append_axes"):
        t = case["batch"] * case["rows"] if op == "norm_rope_axes" else sum(_lengths(case)[1])
        rows = 2 * (hq + hkv) if op == "norm_rope_axes" else 2 * (hq + 2 * hkv)
        angles = min(t, _far(case)) * 4 * case["rot"]
        return {"bytes": t * (rows * row + 4 * case["axes"]) + angles,
                "flops": t * (hq + hkv) * d * 7}
    if op == "diff":
        packed = case["mask"].startswith("document")
        lens = _segments(case) if packed else [case["rows"]] * case["batch"]
        pairs, t = sum(_seen(case, n) for n in lens), sum(lens)
        return {"bytes": t * (2 * (hq + hkv) * row + 8 * hq), "flops": 6.0 * pairs * hq * d}
    if op == "diff_chunk":
        lk, lq = _lengths(case)
        pairs = sum(n * (L - n) + n * (n + 1) // 2 for L, n in zip(lk, lq))
        return {"bytes": sum(lk) * 2 * hkv * row + sum(lq) * hq * (2 * row + 8),
                "flops": 6.0 * pairs * hq * d}
    lk = _decode_lengths(case)
    return {"bytes": sum(lk) * 2 * hkv * row + case["batch"] * hq * (2 * row + 8),
            "flops": 6.0 * sum(lk) * hq * d}


# ------------------------------------------------------------------ inputs

def _int32(values):
    return torch.tensor(values, dtype=torch.int32, device="cuda")


def _cumulative(lens):
    return torch.cat([_int32([0]), _int32(lens).cumsum(0).to(torch.int32)])


def _pages(lk, page, gen):
    """Block table of pages drawn from a shuffled pool with a few spare pages; -1 past the
    last page. Returns (table, num_pages)."""
    per = [-(-L // page) for L in lk]
    num = sum(per) + 7
    perm = torch.randperm(num, generator=gen, device="cuda").to(torch.int32)
    table = torch.full((len(lk), max(1, max(per))), -1, dtype=torch.int32, device="cuda")
    at = 0
    for b, n in enumerate(per):
        table[b, :n] = perm[at:at + n]
        at += n
    return table, num


def _normal(gen, *shape):
    return torch.randn(shape, generator=gen, device="cuda").to(torch.bfloat16)


def _pools(gen, num, hkv, page, d):
    """Page pools of keys and values, made a slice of pages at a time."""
    pools = []
    for _ in range(2):
        pool = torch.empty((num, hkv, page, d), dtype=torch.bfloat16, device="cuda")
        for p0 in range(0, num, 2048):
            pool[p0:p0 + 2048] = _normal(gen, min(2048, num - p0), hkv, page, d)
        pools.append(pool)
    return pools


def _rotation(positions, rot):
    """cos / sin of every position, fp32 [positions, rot]: rot/2 cosines, rot/2 sines. Angles
    in 64 bits: far positions lose them in 32."""
    rate = 10000.0 ** (-torch.arange(0, rot, 2, dtype=torch.float64, device="cuda") / rot)
    angle = torch.arange(positions, dtype=torch.float64, device="cuda")[:, None] * rate
    return torch.cat([angle.cos(), angle.sin()], dim=1).float().contiguous()


def _far(case):
    """Rows of the rotation table: what the positions of _axis_positions reach, or more."""
    most = case["rows"] if case["op"] == "norm_rope_axes" else case["hi"]
    return max(case.get("far", 0), most // (GRID[0] * GRID[1]) + GRID[0] + 1)


def _axis_positions(at, axes, far):
    """Positions int32 [axes, tokens] of tokens at places `at` of videos: frame by frame, each
    frame row by row, all axes going on by one a frame. They end near the table's last row."""
    down, across = GRID
    frame = at // (down * across)
    y, x = at // across % down, at % across
    parts = {2: (y, x), 3: (0 * at, y, x), 4: (0 * at, y, x, (x + y) // 2)}[axes]
    pos = torch.stack([frame + p for p in parts])
    return (pos + max(0, far - 1 - int(pos.max()))).to(torch.int32).contiguous()


def _pair_axis(case):
    """The axis of every rotated pair: a quarter of the pairs for the first axis and the rest in
    runs, or the axes in turns."""
    half, axes = case["rot"] // 2, case["axes"]
    if case["turns"]:
        return [i % axes for i in range(half)]
    first = half // 4
    return [0 if i < first else 1 + (i - first) * (axes - 1) // (half - first)
            for i in range(half)]


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    hq, hkv, d = HEADS[case["heads"]]
    op = case["op"]
    s = {"case": case, "hq": hq, "hkv": hkv, "d": d}
    if op in ("norm_rope_axes", "append_axes"):
        row = d // case["maps"]
        s["maps"], s["rot"], s["interleaved"] = case["maps"], case["rot"], case["interleaved"]
        s["axes"], s["far"] = case["axes"], _far(case)
        s["pair_axis"] = bytes(_pair_axis(case))
        s["cos_sin"] = _rotation(s["far"], case["rot"])
        s["q_weight"] = s["k_weight"] = None
        if case["norm"]:
            s["q_weight"] = 1 + 0.2 * torch.randn(row, generator=gen, device="cuda")
            s["k_weight"] = 1 + 0.2 * torch.randn(row, generator=gen, device="cuda")
    if op == "norm_rope_axes":
        total = s["total"] = case["batch"] * case["rows"]
        s["rows"] = case["rows"]
        s["qkv"] = _normal(gen, total, (hq + 2 * hkv) * d)
        # prompts begin anywhere in a video; single tokens stand anywhere in the table
        most = GRID[0] * GRID[1] * (s["far"] - GRID[0]) if case["rows"] == 1 else case["rows"]
        at = torch.randint(most, (total if case["rows"] == 1 else 1,), generator=gen, device="cuda")
        if case["rows"] > 1:
            at = (at + torch.arange(total, device="cuda")) % case["rows"]
        s["positions"] = _axis_positions(at, s["axes"], s["far"])
        s["q_out"] = torch.empty((case["batch"], hq, case["rows"], d), dtype=torch.bfloat16,
                                 device="cuda")
        s["k_out"] = torch.empty((case["batch"], hkv, case["rows"], d), dtype=torch.bfloat16,
                                 device="cuda")
        return s
    if op == "append_axes":
        lk, lq = _lengths(case)
        total = s["total"] = sum(lq)
        s["page"] = case["page"]
        s["table"], s["num"] = _pages(lk, case["page"], gen)
        s["lk"], s["lq"], s["cu"] = _int32(lk), _int32(lq), _cumulative(lq)
        # q of a step of single tokens goes to decode's [B, Hq, 1, d], of chunks to
        # [1, Hq, total, d]
        s["rows"] = 1 if case["new"] <= 1 else total
        s["qkv"] = _normal(gen, total, (hq + 2 * hkv) * d)
        s["positions"] = _axis_positions(_new_tokens(s)[1], s["axes"], s["far"])
        s["q_out"] = torch.empty((total // s["rows"], hq, s["rows"], d), dtype=torch.bfloat16,
                                 device="cuda")
        s["k_pool"], s["v_pool"] = _pools(gen, s["num"], hkv, case["page"], d)
        return s
    s["lam"] = 0.2 + 0.7 * torch.rand(hq, generator=gen, device="cuda")
    s["weight"] = None
    if case["norm"]:
        s["weight"] = 1 + 0.2 * torch.randn(d, generator=gen, device="cuda")
    s["scale"] = (d // 2) ** -0.5
    if op == "diff":
        s["cu"] = None
        b, n = case["batch"], case["rows"]
        if case["mask"].startswith("document"):
            lens = s["lens"] = _segments(case)
            s["cu"] = _cumulative(lens)
            b, n = 1, sum(lens)
        s["q"], s["k"], s["v"] = (_normal(gen, b, h, n, d) for h in (hq, hkv, hkv))
        s["lse"] = torch.empty((b, hq, 2, n), device="cuda")
    else:
        if op == "diff_chunk":
            lk, lq = _lengths(case)
            s["lq"], s["cu"], s["total"] = lq, _cumulative(lq), sum(lq)
            s["q"] = _normal(gen, 1, hq, sum(lq), d)
            s["lse"] = torch.empty((1, hq, 2, sum(lq)), device="cuda")
        else:
            lk = _decode_lengths(case)
            s["N"] = max(1, max(lk))
            s["cu"] = _cumulative(lk)
            s["q"] = _normal(gen, case["batch"], hq, 1, d)
            s["lse"] = torch.empty((case["batch"], hq, 2), device="cuda")
        s["lk"], s["d_lk"] = lk, _int32(lk)
        s["page"] = case["page"]
        s["table"], s["num"] = _pages(lk, case["page"], gen)
        s["k"], s["v"] = _pools(gen, s["num"], hkv, case["page"], d)
    s["o"] = torch.empty_like(s["q"])
    return s


# ------------------------------------------------------------------ one pass

def run(s):
    if own:
        return _run_own(s, s["case"]["op"])
    return {"norm_rope_axes": _plain_norm_rope, "append_axes": _plain_append, "diff": _plain_diff,
            "diff_chunk": _plain_chunk, "diff_decode": _plain_decode}[s["case"]["op"]](s)


def _run_own(s, op):
    from tiled_attention_gb300 import attn
    hq, hkv, d = s["hq"], s["hkv"], s["d"]
    if op in ("norm_rope_axes", "append_axes"):
        qkv, width = s["qkv"], (hq + 2 * hkv) * d
        q, k, v = qkv[:, :hq * d], qkv[:, hq * d:(hq + hkv) * d], qkv[:, (hq + hkv) * d:]
    if op == "norm_rope_axes":
        attn.check(attn.attn_norm_rope_axes(
            q, k, s["q_out"], s["k_out"], s["total"], s["rows"], hq, hkv, d, s["maps"], width,
            width, s["q_weight"], s["k_weight"], EPS, s["cos_sin"], s["far"], s["rot"],
            s["interleaved"], s["axes"], s["pair_axis"], s["positions"]))
        return {"q": s["q_out"], "k": s["k_out"]}
    if op == "append_axes":
        attn.check(attn.attn_append_paged_axes(
            q, k, v, s["q_out"], s["k_pool"], s["v_pool"], s["case"]["batch"], hq, hkv, s["total"],
            s["rows"], d, s["maps"], width, width, width, s["q_weight"], s["k_weight"], EPS,
            s["cos_sin"], s["far"], s["rot"], s["interleaved"], s["axes"], s["pair_axis"],
            s["positions"], s["cu"], s["lk"], s["table"], s["table"].shape[1], s["page"],
            s["num"]))
        return {"q": s["q_out"], "k": s["k_pool"], "v": s["v_pool"]}
    if op == "diff":
        kind = {"none": attn.ATTN_MASK_NONE, "causal": attn.ATTN_MASK_CAUSAL,
                "sliding": attn.ATTN_MASK_SLIDING, "sliding_bidir": attn.ATTN_MASK_SLIDING_BIDIR,
                "prefix": attn.ATTN_MASK_PREFIX_LM, "document": attn.ATTN_MASK_DOCUMENT,
                "document_bidir": attn.ATTN_MASK_DOCUMENT_BIDIR}[s["case"]["mask"]]
        attn.check(attn.attn_fwd_diff(
            s["q"], s["k"], s["v"], s["o"], s["lse"], s["lam"], s["case"]["batch"], hq, hkv,
            s["q"].shape[2], d, s["scale"], kind, s["case"]["window"], s["cu"], s["weight"], EPS,
            OUT_SCALE))
    elif op == "diff_chunk":
        attn.check(attn.attn_fwd_diff_paged_prefill(
            s["q"], s["k"], s["v"], s["o"], s["lse"], s["lam"], s["case"]["batch"], hq, hkv,
            s["total"], d, s["scale"], s["weight"], EPS, OUT_SCALE, s["cu"], s["d_lk"], s["table"],
            s["table"].shape[1], s["page"], s["num"]))
    else:
        if "workspace" not in s:  # kept with the state, as a serving loop keeps it
            n = attn.attn_workspace_bytes_diff(s["case"]["batch"], hq, hkv, s["N"], d)
            s["workspace"] = torch.empty(max(n, 16), dtype=torch.uint8, device="cuda")
        attn.check(attn.attn_fwd_diff_paged_decode(
            s["q"], s["k"], s["v"], s["o"], s["lse"], s["lam"], s["case"]["batch"], hq, hkv,
            s["N"], d, s["scale"], s["weight"], EPS, OUT_SCALE, s["cu"], s["table"], s["page"],
            s["num"], s["workspace"]))
    return {"o": s["o"], "lse": s["lse"]}


# ------------------------------------------------------------------ plain forms (32 bits)

def _prepared(s, first, heads, weight, pos):
    """Heads first .. first + heads of the projection, normed and turned, fp32 [total, heads,
    d]."""
    d, maps = s["d"], s["maps"]
    x = s["qkv"][:, first * d:(first + heads) * d].float().view(-1, heads * maps, d // maps)
    if weight is not None:
        x = x * ((x * x).mean(dim=-1, keepdim=True) + EPS).rsqrt() * weight
    half = s["rot"] // 2
    axis = torch.tensor(list(s["pair_axis"]), device="cuda")
    at = pos.long()[axis]                                        # [pairs, total]
    i = torch.arange(half, device="cuda")
    cos = s["cos_sin"][at.T, i][:, None, :]
    sin = s["cos_sin"][at.T, half + i][:, None, :]
    out = x.clone()
    if s["interleaved"]:
        a, b = x[..., 0:2 * half:2], x[..., 1:2 * half:2]
        out[..., 0:2 * half:2] = a * cos - b * sin
        out[..., 1:2 * half:2] = b * cos + a * sin
    else:
        a, b = x[..., :half], x[..., half:2 * half]
        out[..., :half] = a * cos - b * sin
        out[..., half:2 * half] = b * cos + a * sin
    return out.view(-1, heads, d)


def _head_major(x, rows):
    """[total, heads, d] to bf16 [total / rows, heads, rows, d]."""
    total, heads, d = x.shape
    return x.view(total // rows, rows, heads, d).transpose(1, 2).to(torch.bfloat16).contiguous()


def _plain_norm_rope(s):
    q = _prepared(s, 0, s["hq"], s["q_weight"], s["positions"])
    k = _prepared(s, s["hq"], s["hkv"], s["k_weight"], s["positions"])
    return {"q": _head_major(q, s["rows"]), "k": _head_major(k, s["rows"])}


def _new_tokens(s):
    """(sequence, place in its context, physical page) of every new token."""
    seq = torch.repeat_interleave(torch.arange(len(s["lq"]), device="cuda"), s["lq"].long(),
                                  output_size=s["total"])
    t = torch.arange(s["total"], device="cuda") - s["cu"].long()[seq]
    at = (s["lk"] - s["lq"]).long()[seq] + t
    return seq, at, s["table"].long()[seq, at // s["page"]]


def _plain_append(s):
    _, at, phys = _new_tokens(s)
    hq, hkv, d = s["hq"], s["hkv"], s["d"]
    q = _prepared(s, 0, hq, s["q_weight"], s["positions"])
    k = _prepared(s, hq, hkv, s["k_weight"], s["positions"])
    slot = at % s["page"]
    s["k_pool"][phys, :, slot] = k.to(torch.bfloat16)
    s["v_pool"][phys, :, slot] = s["qkv"][:, (hq + hkv) * d:].view(-1, hkv, d)
    return {"q": _head_major(q, s["rows"]), "k": s["k_pool"], "v": s["v_pool"]}


def _plain_rows(s, q, k, v, here, lam):
    """Differential attention of fp32 q [..., G, n, d] over k, v [..., 1, m, d] where `here`
    [n, m] (None: everywhere); lam [..., G, 1, 1]. Returns (O fp32, LSE [..., G, 2, n])."""
    half = s["d"] // 2
    parts, lse = [], []
    for m in range(2):
        cut = slice(m * half, (m + 1) * half)
        score = (q[..., cut] * s["scale"]) @ k[..., cut].transpose(-1, -2)
        if here is not None:
            score = score.masked_fill_(~here, -math.inf)
        top = score.amax(dim=-1, keepdim=True).clamp_(min=-3e38)
        p = score.sub_(top).exp_()
        total = p.sum(dim=-1, keepdim=True)
        parts.append((p @ v) / total.clamp(min=1e-38))
        lse.append(torch.where(total > 0, top + total.log(), -math.inf).squeeze(-1))
        del score, p
    y = parts[0] - lam * parts[1]
    if s["weight"] is not None:
        y = y * ((y * y).mean(dim=-1, keepdim=True) + EPS).rsqrt() * s["weight"]
    return y * OUT_SCALE, torch.stack(lse, dim=-2)


def _visible(case, n):
    """Truth values [n, n] of a dense or document mask; None for no mask."""
    mask, w = case["mask"], case["window"]
    if mask in ("none", "document_bidir"):
        return None
    i = torch.arange(n, device="cuda")[:, None]
    j = torch.arange(n, device="cuda")
    if mask == "sliding":
        return (j <= i) & (j > i - w)
    if mask == "sliding_bidir":
        return (j - i).abs() <= w
    if mask == "prefix":
        return (j <= i) | (j < w)
    return j <= i


def _plain_diff(s):
    hq, hkv = s["hq"], s["hkv"]
    g = hq // hkv
    lens = s["lens"] if s["cu"] is not None else [s["q"].shape[2]]
    o, lse = torch.empty_like(s["q"]), torch.empty_like(s["lse"])
    t0 = 0
    for n in lens:
        here = _visible(s["case"], n)
        cut = slice(t0, t0 + n)
        for b in range(s["q"].shape[0]):
            for h in range(hkv):
                heads = slice(h * g, (h + 1) * g)
                y, e = _plain_rows(s, s["q"][b, heads, cut].float(), s["k"][b, h:h + 1, cut].float(),
                                   s["v"][b, h:h + 1, cut].float(), here,
                                   s["lam"][heads].view(g, 1, 1))
                o[b, heads, cut], lse[b, heads, :, cut] = y.to(torch.bfloat16), e
        t0 += n
    return {"o": o, "lse": lse}


def _context(s, b, n):
    """Keys and values of sequence b's first n places, fp32 [Hkv, 1, n, d]."""
    pages = s["table"][b, :-(-n // s["page"])].long()
    return [p[pages].transpose(0, 1).flatten(1, 2)[:, None, :n].float() for p in (s["k"], s["v"])]


def _plain_chunk(s):
    hq, hkv, d = s["hq"], s["hkv"], s["d"]
    g = hq // hkv
    o, lse = torch.empty_like(s["q"]), torch.empty_like(s["lse"])
    t0 = 0
    for b, (L, n) in enumerate(zip(s["lk"], s["lq"])):
        k, v = _context(s, b, L)
        here = (torch.arange(L, device="cuda")
                <= torch.arange(L - n, L, device="cuda")[:, None])
        q = s["q"][0, :, t0:t0 + n].float().view(hkv, g, n, d)
        y, e = _plain_rows(s, q, k, v, here, s["lam"].view(hkv, g, 1, 1))
        o[0, :, t0:t0 + n] = y.view(hq, n, d).to(torch.bfloat16)
        lse[0, :, :, t0:t0 + n] = e.reshape(hq, 2, n)
        t0 += n
    return {"o": o, "lse": lse}


def _plain_decode(s):
    hq, hkv, d = s["hq"], s["hkv"], s["d"]
    g = hq // hkv
    n, cols = s["table"].shape
    keys = cols * s["page"]
    pages = s["table"].long().clamp(min=0)
    k, v = (p[pages].transpose(1, 2).reshape(n, hkv, keys, d).float() for p in (s["k"], s["v"]))
    here = torch.arange(keys, device="cuda").view(1, 1, 1, keys) < s["d_lk"].view(n, 1, 1, 1)
    q = s["q"].float().view(n, hkv, g, d)
    y, e = _plain_rows(s, q, k, v, here, s["lam"].view(hkv, g, 1))
    return {"o": y.view(n, hq, 1, d).to(torch.bfloat16),
            "lse": e.transpose(-1, -2).reshape(n, hq, 2)}


# ------------------------------------------------------------------ definitions (64 bits)

def exact(case, seed):
    s = prepare(case, seed)
    op, hq, hkv, d = case["op"], s["hq"], s["hkv"], s["d"]
    if op == "diff":
        o = torch.empty(s["q"].shape, dtype=torch.float64, device="cuda")
        lse = torch.empty(s["lse"].shape, dtype=torch.float64, device="cuda")
        ends = [s["q"].shape[2]] if s["cu"] is None else s["cu"].tolist()[1:]
        for b in range(s["q"].shape[0]):
            for h in range(hq):
                start = 0
                for end in ends:
                    at = slice(start, end)
                    o[b, h, at], lse[b, h, :, at] = _exact_head(
                        s, h, s["q"][b, h, at], s["k"][b, h * hkv // hq, at],
                        s["v"][b, h * hkv // hq, at], lambda i, n=end - start: _exact_range(
                            case, i, n))
                    start = end
        return {"o": o, "lse": lse}
    if op in ("diff_chunk", "diff_decode"):
        return _exact_paged(s, op == "diff_decode")
    total = s["total"]
    x = s["qkv"].double().view(total, hq + 2 * hkv, d)
    q = _exact_turn(s, x[:, :hq], s["q_weight"])
    k = _exact_turn(s, x[:, hq:hq + hkv], s["k_weight"])
    q = q.reshape(total // s["rows"], s["rows"], hq, d).permute(0, 2, 1, 3)
    if op == "norm_rope_axes":
        return {"q": q, "k": k.reshape(-1, s["rows"], hkv, d).permute(0, 2, 1, 3)}
    where = []
    lk, lq, table = s["lk"].tolist(), s["lq"].tolist(), s["table"].tolist()
    for b in range(len(lk)):
        for p in range(lk[b] - lq[b], lk[b]):
            where.append(table[b][p // s["page"]] * s["page"] + p % s["page"])
    where = torch.tensor(where, device="cuda")
    return {"q": q, "k": _exact_put(s["k_pool"].double(), where, k),
            "v": _exact_put(s["v_pool"].double(), where, x[:, hq + hkv:])}


def _exact_turn(s, x, weight):
    """Norm of each map's row, then each pair as a complex number times cos + i sin."""
    total, heads, d = x.shape
    row = d // s["maps"]
    x = x.reshape(total, heads, s["maps"], row)
    if weight is not None:
        x = x / torch.sqrt(x.pow(2).sum(-1, keepdim=True) / row + EPS) * weight.double()
    half = s["rot"] // 2
    y = x.clone()
    for i, axis in enumerate(s["pair_axis"]):
        angle = s["cos_sin"].double()[s["positions"][axis].long()]
        turn = torch.complex(angle[:, i], angle[:, half + i])[:, None, None]
        a, b = (2 * i, 2 * i + 1) if s["interleaved"] else (i, i + half)
        z = torch.complex(x[..., a], x[..., b]) * turn
        y[..., a], y[..., b] = z.real, z.imag
    return y.view(total, heads, d)


def _exact_put(pool, where, rows):
    """Rows [tokens, Hkv, d] to flat token slots of a pool [num, Hkv, page, d]."""
    num, hkv, page, d = pool.shape
    flat = pool.permute(0, 2, 1, 3).reshape(num * page, hkv, d)
    flat[where] = rows
    return flat.view(num, page, hkv, d).permute(0, 2, 1, 3).contiguous()


def _exact_range(case, i, n):
    """First and last visible key of rows i (a tensor) of a sequence of n tokens."""
    mask, w = case["mask"], case["window"]
    lo, hi = torch.zeros_like(i), torch.full_like(i, n - 1)
    if mask in ("sliding", "sliding_bidir"):
        lo = (i - w + (mask == "sliding")).clamp(min=0)
    if mask in ("causal", "sliding", "document"):
        hi = i
    if mask == "sliding_bidir":
        hi = (i + w).clamp(max=n - 1)
    if mask == "prefix":
        hi = torch.maximum(i, torch.full_like(i, min(w, n) - 1))
    return lo, hi


def _exact_head(s, h, q, k, v, visible):
    """One head over one sequence: q [n, d], k, v [m, d]; `visible` gives the first and last
    visible keys of rows."""
    n, d = q.shape
    q, k, v = q.double(), k.double(), v.double()
    o = torch.empty((n, d), dtype=torch.float64, device="cuda")
    lse = torch.empty((2, n), dtype=torch.float64, device="cuda")
    for r0 in range(0, n, 1024):
        i = torch.arange(r0, min(n, r0 + 1024), device="cuda")
        lo, hi = visible(i)
        j0, j1 = int(lo.min()), int(hi.max()) + 1
        j = torch.arange(j0, j1, device="cuda")
        hide = (j < lo[:, None]) | (j > hi[:, None])
        y = 0.0
        for m, sign in ((0, 1.0), (1, -float(s["lam"][h]))):
            qm, km = (t.view(-1, 2, d // 2)[:, m] for t in (q[r0:r0 + 1024], k[j0:j1]))
            score = torch.where(hide, -math.inf, torch.einsum("id,jd->ij", qm, km) * s["scale"])
            lse[m, r0:r0 + 1024] = torch.logsumexp(score, dim=-1)
            y = y + sign * (torch.softmax(score, dim=-1) @ v[j0:j1])
        o[r0:r0 + 1024] = _exact_out(s, y)
    return o, lse


def _exact_out(s, y):
    if s["weight"] is not None:
        y = y / torch.sqrt(y.pow(2).sum(-1, keepdim=True) / s["d"] + EPS) * s["weight"].double()
    return OUT_SCALE * y


def _exact_paged(s, decode):
    hq, hkv, d, page = s["hq"], s["hkv"], s["d"], s["page"]
    o = torch.zeros(s["q"].shape, dtype=torch.float64, device="cuda")
    lse = torch.full(s["lse"].shape, -math.inf, dtype=torch.float64, device="cuda")
    t0 = 0
    for b, n in enumerate(s["lk"]):
        new = 1 if decode else s["lq"][b]
        if not n:
            continue
        pages = s["table"][b, :-(-n // page)].long()
        k, v = (p[pages].permute(1, 0, 2, 3).reshape(hkv, -1, d)[:, :n] for p in (s["k"], s["v"]))
        if decode:
            q = s["q"][b, :, 0].double().view(hkv, hq // hkv, 2, d // 2)
            score = torch.einsum("hgmd,hnmd->hgmn", q,
                                 k.double().view(hkv, n, 2, d // 2)) * s["scale"]
            lse[b] = torch.logsumexp(score, dim=-1).view(hq, 2)
            a = torch.einsum("hgmn,hnd->hgmd", torch.softmax(score, dim=-1), v.double())
            y = a[:, :, 0].reshape(hq, d) - s["lam"].double()[:, None] * a[:, :, 1].reshape(hq, d)
            o[b, :, 0] = _exact_out(s, y)
            continue
        for h in range(hq):
            o[0, h, t0:t0 + new], lse[0, h, :, t0:t0 + new] = _exact_head(
                s, h, s["q"][0, h, t0:t0 + new], k[h * hkv // hq], v[h * hkv // hq],
                lambda i, first=n - new: (torch.zeros_like(i), i + first))
        t0 += new
    return {"o": o, "lse": lse}
