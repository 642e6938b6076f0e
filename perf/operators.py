"""What the cache operators are measured on: cases, inputs, plain forms and definitions.

The operators prepare queries and keys and keep a paged cache:

  norm_rope    per-head RMS norm of q and k with the position rotation, from the projection's
               token-major layout into the layout attention reads
  append       new tokens' keys and values into bf16 page pools, normed and rotated on the way
  append_fp4   the same into 4-bit page pools; its result is read back as bf16 pages, as
               chunked prefill does next
  unpack_fp4   4-bit pages to bf16 pages
  decode_fp4   paged decode over the 4-bit cache

4-bit pools: uint8 [num_pages, Hkv, page * (d/2 + d/16)]. One (page, kv head) block holds the
codes of its tokens, d/2 bytes each (channel 2c in the low nibble of byte c, E2M1), then their
scales, d/16 bytes each (E4M3, one per 16 channels). A value is code * scale * the tensor's
scale.
"""
import math

import torch

own = False

# Hq, Hkv, d of this repository's configurations: the headline's grouped heads, the document
# workload's d = 64, and its decode's largest group.
HEADS = {"gqa": (32, 8, 128), "mha64": (16, 16, 64), "wide": (64, 4, 64), "mqa": (12, 1, 128)}
EPS = 1e-6
E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)


def listed():
    return [
        # four sequences' next tokens: the smallest call, one launch's latency
        {"name": "norm_rope_step", "op": "norm_rope", "heads": "gqa", "batch": 4, "rows": 1,
         "far": 16384, "rot": 128, "interleaved": False, "norm": True, "given": True},
        # the headline prompt: 2 x 8192 tokens, positions counted from each row's start
        {"name": "norm_rope_prompt", "op": "norm_rope", "heads": "gqa", "batch": 2, "rows": 8192,
         "far": 8192, "rot": 128, "interleaved": False, "norm": True, "given": False},
        # one decode step of 32 sequences: 32 tokens scattered to 32 pages
        {"name": "append_step", "op": "append", "heads": "gqa", "batch": 32, "lo": 256,
         "hi": 2048, "new": 1, "page": 64, "rot": 128, "interleaved": False, "norm": True},
        # chunked prefill of 16 sequences, pages of 16 tokens
        {"name": "append_chunks", "op": "append", "heads": "gqa", "batch": 16, "lo": 2048,
         "hi": 6000, "new": 2048, "page": 16, "rot": 128, "interleaved": False, "norm": True},
        # a few odd prompts, d = 64, a quarter of the channels rotated in adjacent pairs
        {"name": "append_odd_d64", "op": "append", "heads": "mha64", "batch": 5, "lo": 37,
         "hi": 901, "new": 701, "page": 32, "rot": 16, "interleaved": True, "norm": False},
        # one decode step into the 4-bit cache
        {"name": "append_fp4_step", "op": "append_fp4", "heads": "gqa", "batch": 32, "lo": 256,
         "hi": 2048, "new": 1, "page": 64, "rot": 128, "interleaved": False},
        # chunks into the 4-bit cache, read back for the chunk's attention
        {"name": "append_fp4_chunks", "op": "append_fp4", "heads": "gqa", "batch": 16, "lo": 2048,
         "hi": 6000, "new": 2048, "page": 16, "rot": 128, "interleaved": False},
        # a short batch's pages
        {"name": "unpack_fp4_short", "op": "unpack_fp4", "heads": "mha64", "batch": 4, "lo": 500,
         "hi": 1501, "page": 16},
        # 16 long contexts
        {"name": "unpack_fp4_long", "op": "unpack_fp4", "heads": "gqa", "batch": 16, "lo": 2048,
         "hi": 16384, "page": 64},
        # one 16K-token sequence: the step's latency
        {"name": "decode_fp4_one", "op": "decode_fp4", "heads": "gqa", "batch": 1, "lo": 16384,
         "hi": 16384, "page": 64, "empty": 0},
        # the decode batch of the paged benchmark: 32 sequences of 1K to 16K tokens
        {"name": "decode_fp4_batch", "op": "decode_fp4", "heads": "gqa", "batch": 32, "lo": 1024,
         "hi": 16384, "page": 64, "empty": 0},
        # 16 query heads a kv head, d = 64, small pages, slots of a padded batch left empty
        {"name": "decode_fp4_wide", "op": "decode_fp4", "heads": "wide", "batch": 48, "lo": 1,
         "hi": 32768, "page": 16, "empty": 3},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    while True:  # nothing larger than the largest listed case
        case = _draw(rng)
        if work(case)["bytes"] < 780e6:
            return case


def _draw(rng):
    op = rng.choice(["norm_rope", "append", "append_fp4", "unpack_fp4", "decode_fp4"])
    heads = rng.choice(sorted(HEADS))
    d = HEADS[heads][2]
    case = {"op": op, "heads": heads}
    if op == "norm_rope":
        total = _log(rng, 1, 16000)
        batch = rng.choice([1, 2, 3, total])
        case.update(batch=batch, rows=max(1, total // batch), far=_log(rng, 2, 100000),
                    rot=rng.choice([16, 32, d // 2, d, d]),
                    interleaved=rng.random() < 0.3, norm=rng.random() < 0.7,
                    given=rng.random() < 0.6)
        return case
    case.update(page=rng.choice([16, 32, 64, 128]))
    if op in ("append", "append_fp4"):
        hi = _log(rng, 8, 6000)
        new = 1 if rng.random() < 0.4 else _log(rng, 2, 2048)
        case.update(batch=_log(rng, 1, 16), lo=max(1, hi // rng.choice([1, 2, 8])), hi=hi,
                    new=new, rot=rng.choice([32, d // 2, d, d]),
                    interleaved=rng.random() < 0.3)
        if op == "append":
            case.update(norm=rng.random() < 0.5)
        return case
    hi = _log(rng, 2, 16384)
    case.update(batch=_log(rng, 1, 16 if op == "unpack_fp4" else 32),
                lo=max(1, hi // rng.choice([1, 4, 16])), hi=hi)
    if op == "decode_fp4":
        case.update(empty=rng.choice([0, 0, 1, 2]))
    return case


# ------------------------------------------------------------------ shapes of a case

def _spread(case, most):
    """Whole numbers from case['lo'] to `most`, one a sequence, spread over the range in an
    order of their own: sizes go by the case alone, values by the seed."""
    n, lo = case["batch"], case["lo"]
    step = (math.sqrt(5) - 1) / 2
    return [lo + int((most - lo + 1) * ((0.5 + i * step) % 1.0)) for i in range(n)]


def _lengths(case):
    """(context lengths, new tokens) of the sequences."""
    lk = _spread(case, case["hi"])
    new = case.get("new", 0)
    if new <= 1:
        return lk, [new] * len(lk)
    step = math.sqrt(2) - 1
    lq = [max(1, int(min(new, L) * (0.125 + 0.875 * ((0.37 + i * step) % 1.0))))
          for i, L in enumerate(lk)]
    return lk, lq


def _decode_lengths(case):
    lk = _spread(case, case["hi"])
    for i in range(case["empty"]):
        if len(lk) > 1:
            lk[(7 * i + 1) % len(lk)] = 0
    return lk


def work(case):
    hq, hkv, d = HEADS[case["heads"]]
    row, row4 = 2 * d, d // 2 + d // 16
    if case["op"] == "norm_rope":
        t = case["batch"] * case["rows"]
        return {"bytes": t * (hq + hkv) * 2 * row + t * 4 * case["rot"],
                "flops": t * (hq + hkv) * d * 7}
    if case["op"] in ("append", "append_fp4"):
        lk, lq = _lengths(case)
        t = sum(lq)
        given = t * (2 * hq + 2 * hkv) * row + t * 4 * case["rot"]
        if case["op"] == "append":
            return {"bytes": given + t * 2 * hkv * row, "flops": t * (hq + 2 * hkv) * d * 7}
        back = sum(_read_back(case, lk))
        return {"bytes": given + t * 2 * hkv * row4 + back * 2 * hkv * (row4 + row),
                "flops": t * (hq + 2 * hkv) * d * 7 + back * 4 * hkv * d}
    if case["op"] == "unpack_fp4":
        t = sum(_spread(case, case["hi"]))
        return {"bytes": t * 2 * hkv * (row4 + row), "flops": t * 4 * hkv * d}
    lk = _decode_lengths(case)
    return {"bytes": sum(lk) * 2 * hkv * row4 + case["batch"] * hq * (2 * row + 4),
            "flops": 4.0 * sum(lk) * hq * d}


def _read_back(case, lk):
    """Tokens read back after an append: whole contexts after chunks, the last page after a
    step of single tokens."""
    if case["new"] > 1:
        return lk
    return [L - (L - 1) // case["page"] * case["page"] for L in lk]


# ------------------------------------------------------------------ inputs

def _int32(values):
    return torch.tensor(values, dtype=torch.int32, device="cuda")


def _pages(case, lk, gen):
    """Block table of pages drawn from a shuffled pool with a few spare pages; -1 past the
    last page. Returns (table, num_pages)."""
    per = [-(-L // case["page"]) for L in lk]
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


def _rotation(positions, rot):
    """cos / sin of every position, fp32 [positions, rot]: rot/2 cosines, rot/2 sines. Angles
    in 64 bits: far positions lose them in 32."""
    rate = 10000.0 ** (-torch.arange(0, rot, 2, dtype=torch.float64, device="cuda") / rot)
    angle = torch.arange(positions, dtype=torch.float64, device="cuda")[:, None] * rate
    return torch.cat([angle.cos(), angle.sin()], dim=1).float().contiguous()


def _pool4(gen, num, hkv, page, d):
    """A 4-bit pool of quantized normal values, made a slice of pages at a time."""
    pool = torch.empty((num, hkv, page * (d // 2 + d // 16)), dtype=torch.uint8, device="cuda")
    for p0 in range(0, num, 1024):
        x = torch.randn((min(1024, num - p0), hkv, page, d), generator=gen, device="cuda")
        codes, scales = _quantize(x, 1.0)
        pool[p0:p0 + 1024] = torch.cat([codes.flatten(2), scales.flatten(2)], dim=2)
    return pool


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    hq, hkv, d = HEADS[case["heads"]]
    s = {"case": case, "hq": hq, "hkv": hkv, "d": d}
    s["e2m1"] = torch.tensor(E2M1 + tuple(-v for v in E2M1), device="cuda")
    if case["op"] in ("norm_rope", "append", "append_fp4"):
        s["rot"], s["interleaved"] = case["rot"], case["interleaved"]
        s["q_weight"] = s["k_weight"] = None
        if case.get("norm"):
            s["q_weight"] = 1 + 0.2 * torch.randn(d, generator=gen, device="cuda")
            s["k_weight"] = 1 + 0.2 * torch.randn(d, generator=gen, device="cuda")
    if case["op"] == "norm_rope":
        total = s["total"] = case["batch"] * case["rows"]
        s["qkv"] = _normal(gen, total, (hq + 2 * hkv) * d)
        s["far"] = max(case["far"], 1 if case["given"] else case["rows"])
        s["cos_sin"] = _rotation(s["far"], case["rot"])
        s["positions"] = None
        if case["given"]:
            s["positions"] = torch.randint(s["far"], (total,), generator=gen, device="cuda",
                                           dtype=torch.int32)
        s["q_out"] = torch.empty((case["batch"], hq, case["rows"], d), dtype=torch.bfloat16,
                                 device="cuda")
        s["k_out"] = torch.empty((case["batch"], hkv, case["rows"], d), dtype=torch.bfloat16,
                                 device="cuda")
        return s
    page = s["page"] = case["page"]
    if case["op"] in ("append", "append_fp4"):
        lk, lq = _lengths(case)
        total = s["total"] = sum(lq)
        s["table"], num = _pages(case, lk, gen)
        s["num"] = num
        s["lk"], s["lq"] = _int32(lk), _int32(lq)
        s["cu"] = torch.cat([_int32([0]), s["lq"].cumsum(0).to(torch.int32)])
        # q of a step of single tokens goes to decode's [B, Hq, 1, d], of chunks to
        # [1, Hq, total, d]
        s["rows"] = 1 if case["new"] <= 1 else total
        s["qkv"] = _normal(gen, total, (hq + 2 * hkv) * d)
        s["far"] = case["hi"]
        s["cos_sin"] = _rotation(s["far"], case["rot"])
        s["q_out"] = torch.empty((total // s["rows"], hq, s["rows"], d), dtype=torch.bfloat16,
                                 device="cuda")
        if case["op"] == "append":
            s["k_pool"] = _normal(gen, num, hkv, page, d)
            s["v_pool"] = _normal(gen, num, hkv, page, d)
            return s
        s["k_pool"], s["v_pool"] = (_pool4(gen, num, hkv, page, d) for _ in range(2))
        s["k_scale"], s["v_scale"] = 0.5, 0.0625
        back = _read_back(case, lk)
        s["back"] = _int32(back)
        s["back_table"] = s["table"]
        if case["new"] <= 1:
            last = _int32([(L - 1) // page for L in lk])
            s["back_table"] = s["table"].gather(1, last[:, None].long()).contiguous()
    elif case["op"] == "unpack_fp4":
        lk = _spread(case, case["hi"])
        s["back_table"], num = _pages(case, lk, gen)
        s["num"], s["back"] = num, _int32(lk)
        s["k_pool"], s["v_pool"] = (_pool4(gen, num, hkv, page, d) for _ in range(2))
        s["k_scale"], s["v_scale"] = 0.5, 0.0625
    else:
        lk = _decode_lengths(case)
        s["N"] = max(1, max(lk))
        s["table"], num = _pages(case, lk, gen)
        s["num"], s["lk"] = num, _int32(lk)
        s["cu"] = torch.cat([_int32([0]), s["lk"].cumsum(0).to(torch.int32)])
        s["k_pool"], s["v_pool"] = (_pool4(gen, num, hkv, page, d) for _ in range(2))
        s["k_scale"], s["v_scale"] = 1.25, 0.0625
        s["q"] = _normal(gen, case["batch"], hq, 1, d)
        s["o"] = torch.empty_like(s["q"])
        s["lse"] = torch.empty((case["batch"], hq), device="cuda")
        return s
    n, cols = s["back_table"].shape
    s["k_back"], s["v_back"] = (torch.zeros((n * cols, hkv, page, d), dtype=torch.bfloat16,
                                            device="cuda") for _ in range(2))
    return s


# ------------------------------------------------------------------ one pass

def run(s):
    op = s["case"]["op"]
    if own:
        return _run_own(s, op)
    if op == "norm_rope":
        return _plain_norm_rope(s)
    if op == "append":
        return _plain_append(s)
    if op == "append_fp4":
        q = _plain_append_fp4(s)
        return {"q": q, **_plain_unpack(s)}
    if op == "unpack_fp4":
        return _plain_unpack(s)
    return _plain_decode(s)


def _run_own(s, op):
    from tiled_attention_gb300 import attn
    hq, hkv, d = s["hq"], s["hkv"], s["d"]
    if op in ("norm_rope", "append", "append_fp4"):
        qkv, width = s["qkv"], (hq + 2 * hkv) * d
        q, k, v = qkv[:, :hq * d], qkv[:, hq * d:(hq + hkv) * d], qkv[:, (hq + hkv) * d:]
    if op == "norm_rope":
        rc = attn.attn_norm_rope(q, k, s["q_out"], s["k_out"], s["total"], s["case"]["rows"], hq,
                                 hkv, d, width, width, s["q_weight"], s["k_weight"], EPS,
                                 s["cos_sin"], s["far"], s["rot"], s["interleaved"],
                                 s["positions"])
        attn.check(rc)
        return {"q": s["q_out"], "k": s["k_out"]}
    if op == "append":
        rc = attn.attn_append_paged(q, k, v, s["q_out"], s["k_pool"], s["v_pool"],
                                    s["case"]["batch"], hq, hkv, s["total"], s["rows"], d, width,
                                    width, width, s["q_weight"], s["k_weight"], EPS,
                                    s["cos_sin"], s["far"], s["rot"], s["interleaved"], s["cu"],
                                    s["lk"], s["table"], s["table"].shape[1], s["page"],
                                    s["num"])
        attn.check(rc)
        return {"q": s["q_out"], "k": s["k_pool"], "v": s["v_pool"]}
    if op == "append_fp4":
        rc = attn.attn_append_paged_fp4(q, k, v, s["q_out"], s["k_pool"], s["v_pool"],
                                        s["k_scale"], s["v_scale"], s["case"]["batch"], hq, hkv,
                                        s["total"], s["rows"], d, width, width, width, None, None,
                                        EPS, s["cos_sin"], s["far"], s["rot"], s["interleaved"],
                                        s["cu"], s["lk"], s["table"], s["table"].shape[1],
                                        s["page"], s["num"])
        attn.check(rc)
    if op in ("append_fp4", "unpack_fp4"):
        n, cols = s["back_table"].shape
        attn.check(attn.attn_unpack_pages_fp4(s["k_pool"], s["k_back"], s["k_scale"],
                                              s["back_table"], s["back"], n, cols, hkv, s["page"],
                                              d, s["num"]))
        attn.check(attn.attn_unpack_pages_fp4(s["v_pool"], s["v_back"], s["v_scale"],
                                              s["back_table"], s["back"], n, cols, hkv, s["page"],
                                              d, s["num"]))
        got = {"k": s["k_back"], "v": s["v_back"]}
        return {"q": s["q_out"], **got} if op == "append_fp4" else got
    if "workspace" not in s:  # kept with the state, as a serving loop keeps it
        n = attn.attn_workspace_bytes_fp4(s["case"]["batch"], hq, hkv, s["N"], d)
        s["workspace"] = torch.empty(max(n, 16), dtype=torch.uint8, device="cuda")
    rc = attn.attn_fwd_paged_decode_fp4(s["q"], s["k_pool"], s["v_pool"], s["o"], s["lse"],
                                        s["case"]["batch"], hq, hkv, s["N"], d, d ** -0.5,
                                        s["k_scale"], s["v_scale"], s["cu"], s["table"],
                                        s["page"], s["num"], s["workspace"])
    attn.check(rc)
    return {"o": s["o"], "lse": s["lse"]}


# ------------------------------------------------------------------ plain forms (32 bits)

def _rows(s, first, heads):
    """Heads first .. first + heads of the projection, fp32 [total, heads, d]."""
    d = s["d"]
    return s["qkv"][:, first * d:(first + heads) * d].float().view(-1, heads, d)


def _norm(x, weight):
    if weight is None:
        return x
    return x * ((x * x).mean(dim=-1, keepdim=True) + EPS).rsqrt() * weight


def _rotate(s, x, positions):
    half = s["rot"] // 2
    cs = s["cos_sin"][positions.long()][:, None, :]
    cos, sin = cs[..., :half], cs[..., half:]
    out = x.clone()
    if s["interleaved"]:
        a, b = x[..., 0:2 * half:2], x[..., 1:2 * half:2]
        out[..., 0:2 * half:2] = a * cos - b * sin
        out[..., 1:2 * half:2] = b * cos + a * sin
    else:
        a, b = x[..., :half], x[..., half:2 * half]
        out[..., :half] = a * cos - b * sin
        out[..., half:2 * half] = b * cos + a * sin
    return out


def _head_major(x, rows):
    """[total, heads, d] to bf16 [total / rows, heads, rows, d]."""
    total, heads, d = x.shape
    return x.view(total // rows, rows, heads, d).transpose(1, 2).to(torch.bfloat16).contiguous()


def _plain_norm_rope(s):
    rows = s["case"]["rows"]
    pos = s["positions"]
    if pos is None:
        pos = torch.arange(s["total"], device="cuda") % rows
    q = _rotate(s, _norm(_rows(s, 0, s["hq"]), s["q_weight"]), pos)
    k = _rotate(s, _norm(_rows(s, s["hq"], s["hkv"]), s["k_weight"]), pos)
    return {"q": _head_major(q, rows), "k": _head_major(k, rows)}


def _new_tokens(s):
    """(sequence, position in its context, physical page) of every new token."""
    seq = torch.repeat_interleave(torch.arange(len(s["lq"]), device="cuda"), s["lq"].long(),
                                  output_size=s["total"])
    t = torch.arange(s["total"], device="cuda") - s["cu"].long()[seq]
    pos = (s["lk"] - s["lq"]).long()[seq] + t
    return seq, pos, s["table"].long()[seq, pos // s["page"]]


def _plain_append(s):
    seq, pos, phys = _new_tokens(s)
    hq, hkv = s["hq"], s["hkv"]
    q = _rotate(s, _norm(_rows(s, 0, hq), s["q_weight"]), pos)
    k = _rotate(s, _norm(_rows(s, hq, hkv), s["k_weight"]), pos)
    slot = pos % s["page"]
    s["k_pool"][phys, :, slot] = k.to(torch.bfloat16)
    s["v_pool"][phys, :, slot] = _rows(s, hq + hkv, hkv).to(torch.bfloat16)
    return {"q": _head_major(q, s["rows"]), "k": s["k_pool"], "v": s["v_pool"]}


def _quantize(x, scale):
    """fp32 [..., d] to (codes uint8 [..., d/2], scales uint8 [..., d/16])."""
    inv = float(torch.tensor(1.0) / torch.tensor(scale, dtype=torch.float32))
    xs = (x * inv).unflatten(-1, (-1, 16))
    sf = (xs.abs().amax(dim=-1) / 6.0).clamp(max=448.0).to(torch.float8_e4m3fn)
    s = sf.float().unsqueeze(-1)
    y = torch.where(s > 0, xs / s, torch.zeros_like(xs))
    a = y.abs()
    # Round to the nearest code, ties to the even one.
    code = ((a > 0.25).to(torch.uint8) + (a >= 0.75) + (a > 1.25) + (a >= 1.75) + (a > 2.5)
            + (a >= 3.5) + (a > 5.0))
    code = (code + 8 * (y < 0)).to(torch.uint8).flatten(-2)
    return code[..., 0::2] | (code[..., 1::2] << 4), sf.view(torch.uint8)


def _plain_append_fp4(s):
    seq, pos, phys = _new_tokens(s)
    hq, hkv, d, page = s["hq"], s["hkv"], s["d"], s["page"]
    slot = pos % page
    q = _rotate(s, _rows(s, 0, hq), pos)
    k = _rotate(s, _rows(s, hq, hkv), pos)
    _write4(s["k_pool"], phys, slot, page, d, *_quantize(k, s["k_scale"]))
    _write4(s["v_pool"], phys, slot, page, d, *_quantize(_rows(s, hq + hkv, hkv), s["v_scale"]))
    return _head_major(q, s["rows"])


def _write4(pool, phys, slot, page, d, codes, scales):
    num, hkv, _ = pool.shape
    pool[:, :, :page * (d // 2)].unflatten(2, (page, d // 2))[phys, :, slot] = codes
    pool[:, :, page * (d // 2):].unflatten(2, (page, d // 16))[phys, :, slot] = scales


def _values(s, pool, pages):
    """Values of whole pages of a 4-bit pool, without the tensor's scale: fp32
    [*pages.shape, Hkv, page, d]."""
    d, page = s["d"], s["page"]
    raw = pool[pages.long().clamp(min=0)]
    codes = raw[..., :page * (d // 2)].unflatten(-1, (page, d // 2))
    both = torch.stack([codes & 15, codes >> 4], dim=-1).flatten(-2)
    sf = raw[..., page * (d // 2):].contiguous().view(torch.float8_e4m3fn).float()
    sf = sf.unflatten(-1, (page, d // 16))
    return (s["e2m1"][both.int()].unflatten(-1, (-1, 16)) * sf.unsqueeze(-1)).flatten(-2)


def _plain_unpack(s):
    n, cols = s["back_table"].shape
    page = s["page"]
    at = torch.arange(cols * page, device="cuda").view(1, cols, 1, page, 1)
    here = at < s["back"].view(n, 1, 1, 1, 1)
    got = {}
    for_k = _values(s, s["k_pool"], s["back_table"]) * s["k_scale"]
    got["k"] = torch.where(here, for_k, 0.0).to(torch.bfloat16).flatten(0, 1)
    del for_k
    for_v = _values(s, s["v_pool"], s["back_table"]) * s["v_scale"]
    got["v"] = torch.where(here, for_v, 0.0).to(torch.bfloat16).flatten(0, 1)
    return got


def _plain_decode(s):
    hkv, d = s["hkv"], s["d"]
    n, cols = s["table"].shape
    group = s["hq"] // hkv
    keys = cols * s["page"]
    q = s["q"].float().view(n, hkv, group, d) * (d ** -0.5 * s["k_scale"])
    k = _values(s, s["k_pool"], s["table"]).transpose(1, 2).reshape(n, hkv, keys, d)
    score = q @ k.transpose(-1, -2)
    del k
    here = torch.arange(keys, device="cuda").view(1, 1, 1, keys) < s["lk"].view(n, 1, 1, 1)
    score = torch.where(here, score, -math.inf)
    top = score.amax(dim=-1, keepdim=True).clamp(min=-3e38)
    p = (score - top).exp()
    total = p.sum(dim=-1, keepdim=True)
    v = _values(s, s["v_pool"], s["table"]).transpose(1, 2).reshape(n, hkv, keys, d)
    o = (p @ v) * (s["v_scale"] / total.clamp(min=1e-38))
    lse = torch.where(total > 0, top + total.log(), -math.inf)
    return {"o": o.view(n, s["hq"], 1, d).to(torch.bfloat16), "lse": lse.view(n, s["hq"])}


# ------------------------------------------------------------------ definitions (64 bits)

def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "decode_fp4":
        return _exact_decode(s)
    if op == "unpack_fp4":
        return _exact_pages(s)
    hq, hkv, d, total = s["hq"], s["hkv"], s["d"], s["total"]
    x = s["qkv"].double().view(total, hq + 2 * hkv, d)
    if op == "norm_rope":
        pos = [i % case["rows"] for i in range(total)]
        pos = torch.tensor(pos, device="cuda") if s["positions"] is None else s["positions"].long()
        rows = case["rows"]
    else:
        pos, where = [], []
        lk, lq, table = s["lk"].tolist(), s["lq"].tolist(), s["table"].tolist()
        for b in range(len(lk)):
            for p in range(lk[b] - lq[b], lk[b]):
                pos.append(p)
                where.append(table[b][p // s["page"]] * s["page"] + p % s["page"])
        pos, where = (torch.tensor(v, device="cuda") for v in (pos, where))
        rows = s["rows"]
    q = _exact_turn(s, x[:, :hq], s["q_weight"], pos)
    k = _exact_turn(s, x[:, hq:hq + hkv], s["k_weight"], pos)
    v = x[:, hq + hkv:]
    q = q.reshape(total // rows, rows, hq, d).permute(0, 2, 1, 3)
    if op == "norm_rope":
        return {"q": q, "k": k.reshape(total // rows, rows, hkv, d).permute(0, 2, 1, 3)}
    if op == "append":
        return {"q": q, "k": _exact_put(s["k_pool"].double(), where, k),
                "v": _exact_put(s["v_pool"].double(), where, v)}
    got = {"q": q}
    for name, y in (("k", k), ("v", v)):
        value = _exact_grid(y / s[name + "_scale"]) * s[name + "_scale"]
        every = _exact_values(s, s[name + "_pool"]) * s[name + "_scale"]
        got[name] = _exact_back(s, _exact_put(every, where, value))
    return got


def _exact_turn(s, x, weight, pos):
    """Norm, then each pair as a complex number times cos + i sin."""
    if weight is not None:
        x = x / torch.sqrt(x.pow(2).sum(-1, keepdim=True) / s["d"] + EPS) * weight.double()
    half = s["rot"] // 2
    i = torch.arange(half, device="cuda")
    first, second = (2 * i, 2 * i + 1) if s["interleaved"] else (i, i + half)
    turn = torch.complex(*(s["cos_sin"].double()[pos].split(half, dim=1)))
    z = torch.complex(x[..., first], x[..., second]) * turn[:, None]
    y = x.clone()
    y[..., first], y[..., second] = z.real, z.imag
    return y


def _exact_put(pool, where, rows):
    """Rows [tokens, Hkv, d] to flat token slots of a pool [num, Hkv, page, d]."""
    num, hkv, page, d = pool.shape
    flat = pool.permute(0, 2, 1, 3).reshape(num * page, hkv, d)
    flat[where] = rows
    return flat.view(num, page, hkv, d).permute(0, 2, 1, 3).contiguous()


def _exact_float(v, digits, low, top):
    """v rounded to nearest even on a float grid: `digits` bits after the leading one, least
    exponent `low`, largest magnitude `top`."""
    m, e = torch.frexp(v)
    e = (e - 1).clamp(min=low)
    step = torch.exp2((e - digits).double())
    return (torch.round(v / step) * step).clamp(-top, top)


def _exact_grid(y):
    """What 4 bits and their scale keep of y [..., d], in 64 bits."""
    block = y.reshape(*y.shape[:-1], -1, 16)
    s = _exact_float(block.abs().amax(-1, keepdim=True) / 6.0, 3, -6, 448.0)
    return torch.where(s > 0, _exact_float(block / torch.where(s > 0, s, 1.0), 1, 0, 6.0) * s,
                       0.0).reshape(y.shape)


def _exact_values(s, pool):
    """A 4-bit pool's values by the formats' bits, without the tensor's scale."""
    d, page = s["d"], s["page"]
    cut = page * d // 2
    c = pool[..., :cut].reshape(*pool.shape[:2], page, d // 2)
    c = torch.stack([c % 16, c // 16], dim=-1).reshape(*pool.shape[:2], page, d).double()
    sign = 1 - 2 * (c >= 8).double()
    e, m = torch.div(c % 8, 2, rounding_mode="floor"), c % 2
    code = sign * torch.where(e > 0, (1 + m / 2) * torch.exp2(e - 1), m / 2)
    b = pool[..., cut:].reshape(*pool.shape[:2], page, d // 16).double()
    e, m = torch.div(b % 128, 8, rounding_mode="floor"), b % 8
    sf = torch.where(e > 0, (1 + m / 8) * torch.exp2(e - 7), m / 8 * 2.0 ** -6)
    return code * sf.repeat_interleave(16, dim=-1)


def _exact_back(s, values):
    """Pages of values as the block table lists them; what lies past a length is zero."""
    table, back, page = s["back_table"].tolist(), s["back"].tolist(), s["page"]
    out = torch.zeros((len(table) * len(table[0]), *values.shape[1:]), dtype=torch.float64,
                      device="cuda")
    for b, row in enumerate(table):
        n = -(-back[b] // page)
        if n:
            out[b * len(row):b * len(row) + n] = values[torch.tensor(row[:n], device="cuda")]
            out[b * len(row) + n - 1, :, back[b] - (n - 1) * page:] = 0
    return out


def _exact_pages(s):
    return {n: _exact_back(s, _exact_values(s, s[n + "_pool"]) * s[n + "_scale"])
            for n in ("k", "v")}


def _exact_decode(s):
    hq, hkv, d = s["hq"], s["hkv"], s["d"]
    lk, table = s["lk"].tolist(), s["table"]
    o = torch.zeros((len(lk), hq, 1, d), dtype=torch.float64, device="cuda")
    lse = torch.full((len(lk), hq), -math.inf, dtype=torch.float64, device="cuda")
    for b, n in enumerate(lk):
        if not n:
            continue
        pages = table[b, :-(-n // s["page"])].long()
        k, v = (_exact_values(s, s[name + "_pool"][pages]).transpose(0, 1)
                .reshape(hkv, -1, d)[:, :n] * s[name + "_scale"] for name in ("k", "v"))
        q = s["q"][b, :, 0].double().view(hkv, hq // hkv, d)
        score = torch.einsum("hgd,hnd->hgn", q, k) * d ** -0.5
        lse[b] = torch.logsumexp(score, dim=-1).view(hq)
        o[b, :, 0] = torch.einsum("hgn,hnd->hgd", torch.softmax(score, dim=-1), v).reshape(hq, d)
    return {"o": o, "lse": lse}
