"""Cases, plain forms and exact values of the operators around the attention
calls: rotary positions with the append, copies of pages, and the verification
of drafted tokens.

Four operators, named by a case's "op":

  rotary   rotary_append_fp8: queries and keys turned by positions on one or
           several axes, keys and values quantised into the paged cache
  embed    rotary_embed: the turn alone, bf16 to bf16 (caches that another
           append fills)
  copy     copy_pages: pages copied within the caches of all layers
  verify   verify_drafts: drafted tokens accepted or replaced, from the
           target's and the draft's probabilities and given random numbers

`own` is set from outside: False runs the plain forms below, True the library's
entry points.
"""
import math

import numpy as np
import torch

own = False

WEIGHT_BITS = 42   # a probability is a whole number of 2^-42 when a token is drawn
UNIFORM_BITS = 24  # and a uniform number one of 2^-24


# ------------------------------------------------------------------ the cases
def listed():
    return [
        # a decode step of 64 requests, text: every axis has the same position
        dict(name="rotary_step_b64", op="rotary", tokens=64, hq=64, hkv=8, dim=128, rot=128, first=0, pairs="halves", axes=3, page=16, gran="tensor", span=32768),
        # the smallest step: 4 requests, 8/2 heads
        dict(name="rotary_step_b4", op="rotary", tokens=4, hq=8, hkv=2, dim=128, rot=128, first=0, pairs="halves", axes=1, page=16, gran="head", span=300),
        # a prompt with images and video frames, one scale per token, far positions
        dict(name="rotary_prompt_16k", op="rotary", tokens=16001, hq=64, hkv=8, dim=128, rot=128, first=0, pairs="halves", axes=3, page=64, gran="token", span=1048576),
        # a chunk over an MLA latent cache: the last 64 of 576 channels turn, as neighbours
        dict(name="rotary_latent_2k", op="rotary", tokens=2039, hq=128, hkv=1, dim=576, rot=64, first=512, pairs="neighbours", axes=1, page=64, gran="tensor", span=65536),
        # queries of a step whose keys go to a cache with scales per block
        dict(name="embed_step_b64", op="embed", tokens=64, hq=64, hkv=0, dim=128, rot=128, first=0, pairs="halves", axes=3, span=32768),
        # queries of a chunk, half of the channels turned
        dict(name="embed_prompt_4k", op="embed", tokens=4099, hq=48, hkv=0, dim=128, rot=64, first=0, pairs="neighbours", axes=2, span=131072),
        # one request forked: its last page in one layer's caches
        dict(name="copy_fork_b1", op="copy", pages=64, pairs=1, layers=1, hkv=8, page=64, gran="block"),
        # 64 requests forked, 32 layers: the last page of each
        dict(name="copy_fork_b64_l32", op="copy", pages=257, pairs=64, layers=32, hkv=8, page=16, gran="token"),
        # a pool compacted: a third of its pages move
        dict(name="copy_compact", op="copy", pages=4099, pairs=1361, layers=1, hkv=8, page=64, gran="block"),
        # one request, a small vocabulary, four drafts
        dict(name="verify_b1_v32k", op="verify", batch=1, max_drafts=4, vocab=32768, dtype="float32", draft=True),
        # 64 requests with up to seven drafts each, an odd vocabulary
        dict(name="verify_b64_v128k", op="verify", batch=64, max_drafts=7, vocab=128259, dtype="float32", draft=True),
        # drafts looked up in the prompt: they have no distribution of their own
        dict(name="verify_b96_lookup", op="verify", batch=96, max_drafts=5, vocab=152064, dtype="bfloat16", draft=False),
    ]


HEADS = [(8, 2), (64, 8), (48, 48), (16, 1), (20, 4), (32, 8), (7, 1), (12, 6)]
PAGES = [16, 32, 48, 64, 96, 128]
# head_dim, channels that turn, the first of them, how they pair
TURNS = [(128, 128, 0, "halves"), (128, 64, 0, "halves"), (128, 64, 0, "neighbours"), (128, 96, 16, "halves"),
         (64, 64, 0, "neighbours"), (256, 64, 0, "halves"), (80, 32, 48, "halves"), (576, 64, 512, "neighbours")]


def _log_uniform(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    """A case of the ranges above: from one token, page or request to the
    largest, odd sizes, every head layout and page size the tests use."""
    op = rng.choice(["rotary", "embed", "copy", "verify"])
    if op == "verify":
        batch = _log_uniform(rng, 1, 256)
        drafts = rng.randint(0, 8)
        # no more rows times words than the largest listed case
        room = 64 * 5 * 128259 // (batch * (drafts + 1))
        vocab = _log_uniform(rng, min(1000, room), min(262144, room))
        return dict(op=op, batch=batch, max_drafts=drafts, vocab=vocab, dtype=rng.choice(["float32", "float32", "bfloat16", "float16"]),
                    draft=rng.random() < 0.7)
    if op == "copy":
        hkv, page = rng.choice([1, 2, 4, 6, 8, 48]), rng.choice(PAGES)
        layers = _log_uniform(rng, 1, 48)
        room = (1 << 29) // (layers * hkv * page * 128)   # pages in K and as many in V
        pages = _log_uniform(rng, min(4, room), min(8192, room))
        return dict(op=op, pages=pages, pairs=_log_uniform(rng, 1, pages // 3), layers=layers, hkv=hkv, page=page,
                    gran=rng.choice(["tensor", "token", "block"]))
    hq, hkv = rng.choice(HEADS)
    dim, rot, first, pairs = rng.choice(TURNS)
    axes = rng.choice([1, 1, 2, 3])
    if dim == 576:
        hq, hkv = rng.choice([128, 64, 16]), 1
    room = 16001 * 80 * 128 // ((hq + 2 * hkv) * dim)
    case = dict(op=op, tokens=_log_uniform(rng, 1, min(16384, room)), hq=hq, hkv=hkv, dim=dim, rot=rot, first=first, pairs=pairs,
                axes=axes, span=_log_uniform(rng, 256, 1 << 20))
    if op == "rotary":
        case.update(page=rng.choice(PAGES), gran=rng.choice(["tensor", "head"] if dim == 576 else ["tensor", "head", "token"]))
    else:
        case["hkv"] = 0
    return case


def _has_v(case):
    return case["dim"] != 576   # the latent cache is key and value at once


def _counts(case):
    """Query tokens of each request: the last known token and 0 to max_drafts
    drafted ones."""
    return [1 + (3 * i + case["max_drafts"]) % (case["max_drafts"] + 1) for i in range(case["batch"])]


def _row_bytes(case):
    """Bytes of a page in each array of one layer: K, V and their scales."""
    kv = case["hkv"] * case["page"] * 128
    scale = {"tensor": 0, "token": 4 * case["hkv"] * case["page"], "block": 4 * case["hkv"]}[case["gran"]]
    return 2 * (kv + scale)


def work(case):
    op = case["op"]
    if op == "copy":
        return {"bytes": 2 * case["pairs"] * case["layers"] * _row_bytes(case) + 8 * case["pairs"], "flops": 0}
    if op == "verify":
        size = {"float32": 4, "bfloat16": 2, "float16": 2}[case["dtype"]]
        # one row of the target's for every request; one of the draft's for those with drafts (none where all are
        # accepted, which the inputs decide)
        rows = case["batch"] + (sum(n > 1 for n in _counts(case)) if case["draft"] else 0)
        return {"bytes": rows * case["vocab"] * size + 12 * sum(_counts(case)), "flops": 3 * rows * case["vocab"]}
    t, dim, rot = case["tokens"], case["dim"], case["rot"]
    q = t * case["hq"] * dim * 4
    if op == "embed":
        return {"bytes": q + 4 * t * case["axes"], "flops": 3 * t * case["hq"] * rot}
    kv = t * case["hkv"] * dim * (2 if _has_v(case) else 1)
    scales = 4 * t * case["hkv"] * 2 if case["gran"] == "token" else 0
    return {"bytes": q + 3 * kv + scales + t * (8 + 4 * case["axes"]), "flops": 3 * t * (case["hq"] + case["hkv"]) * rot + kv}


# --------------------------------------------------------------------- inputs
def _generator(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _normal(shape, g):
    """Normal values with a few larger channels, as projections give them."""
    gain = torch.ones(shape[-1], device="cuda")
    gain[torch.randint(0, shape[-1], (4,), device="cuda", generator=g)] = 4.0
    out = torch.empty(shape, dtype=torch.bfloat16, device="cuda")
    for part, to in zip(range(0, shape[0], 4096), out.split(4096)):
        to.copy_(torch.randn(to.shape, device="cuda", generator=g) * gain)
    return out


def _positions(case, rng):
    """int32 [axes][tokens]: text counts up on every axis alike; between texts
    stand pictures, whose tokens share the first axis and run over a grid of
    rows and columns on the others."""
    t, axes, span = case["tokens"], case["axes"], case["span"]
    if t <= 64 or axes == 1:   # a step: one token of each request; or text alone
        start = rng.integers(0, span, t) if t <= 64 else rng.integers(0, max(1, span - t)) + np.arange(t)
        return np.repeat(start[None], axes, 0).astype(np.int32)
    got, at = [], int(rng.integers(0, max(1, span - t)))
    while sum(x.shape[1] for x in got) < t:
        n = int(rng.integers(16, 512))
        got.append(np.repeat(at + np.arange(n)[None], axes, 0))
        at += n
        rows, cols = (int(x) for x in rng.integers(4, 40, 2))
        grid = [np.zeros(rows * cols), np.repeat(np.arange(rows), cols), np.tile(np.arange(cols), rows)]
        got.append(at + np.stack(grid[:axes]).astype(np.int64))
        at += max(rows, cols)
    return np.concatenate(got, 1)[:, :t].astype(np.int32)


def _frequencies(case):
    """Radians per position of each pair, and the axis it follows: a stretch of
    the pairs for each axis."""
    half = case["rot"] // 2
    i = np.arange(half)
    return 500000.0 ** (-i / half), (i * case["axes"] // half).astype(np.int32)


def prepare(case, seed):
    g, rng = _generator(seed), np.random.default_rng(seed)
    op = case["op"]
    s = dict(case=case)
    if op in ("rotary", "embed"):
        t, dim = case["tokens"], case["dim"]
        s["positions"] = torch.from_numpy(_positions(case, rng)).cuda()
        s["frequencies"], s["axes"] = _frequencies(case)
        s["frequency"], s["axis"] = torch.from_numpy(s["frequencies"]).cuda(), torch.from_numpy(s["axes"]).cuda().long()
        s["q"] = _normal((t, case["hq"], dim), g)
        s["q_out"] = torch.empty_like(s["q"])
        if op == "embed":
            return s
        pages = -(-t // case["page"]) + 3
        slots = rng.permutation(pages)[np.arange(t) // case["page"]] * case["page"] + np.arange(t) % case["page"]
        slots[rng.random(t) < 0.01] = -1   # padding of the batch
        s["slots"] = torch.from_numpy(slots.astype(np.int64)).cuda()
        hkv, gran = case["hkv"], case["gran"]
        for x in "kv" if _has_v(case) else "k":
            s[x + "_new"] = _normal((t, hkv, dim), g)
            s[x + "_cache"] = torch.randint(0, 120, (pages, hkv, case["page"], dim), dtype=torch.uint8, device="cuda", generator=g)
            if gran == "token":
                s[x + "_scales"] = torch.rand((pages, hkv, case["page"]), device="cuda", generator=g)
            else:
                s[x + "_scales"] = torch.rand(hkv if gran == "head" else 1, device="cuda", generator=g) * 0.02 + 0.03
        return s
    if op == "copy":
        layers, pages, hkv, page = case["layers"], case["pages"], case["hkv"], case["page"]
        for x in "kv":
            s[x + "_cache"] = torch.randint(0, 120, (layers, pages, hkv, page, 128), dtype=torch.uint8, device="cuda", generator=g)
            if case["gran"] != "tensor":
                shape = (layers, pages, hkv, page) if case["gran"] == "token" else (layers, pages, hkv)
                s[x + "_scales"] = torch.rand(shape, device="cuda", generator=g)
        ids, n = rng.permutation(pages), case["pairs"]
        # a fork may copy one page to several; a page is written once and never read then
        s["pairs"] = torch.from_numpy(np.stack([rng.choice(ids[n:], n), ids[:n]], 1).astype(np.int32)).cuda()
        return s
    vocab, dtype = case["vocab"], getattr(torch, case["dtype"])
    counts = _counts(case)
    rows = sum(counts)
    s["q_start"] = torch.from_numpy(np.concatenate([[0], np.cumsum(counts)]).astype(np.int32)).cuda()
    s["target"] = torch.empty((rows, vocab), dtype=dtype, device="cuda")
    s["draft"] = torch.empty((rows, vocab), dtype=dtype, device="cuda") if case["draft"] else None
    tokens = torch.zeros(rows, dtype=torch.int64, device="cuda")
    for lo in range(0, rows, 64):
        hi = min(rows, lo + 64)
        logits = torch.randn((hi - lo, vocab), device="cuda", generator=g) * 3
        s["target"][lo:hi] = torch.softmax(logits, 1)
        guess = torch.softmax(logits + torch.randn(logits.shape, device="cuda", generator=g) * 0.7, 1)
        if case["draft"]:
            s["draft"][lo:hi] = guess
        # the token after each row, drawn from the draft's distribution (by exponential waiting times)
        wait = torch.empty_like(guess).exponential_(generator=g)
        tokens[lo:hi] = (guess / wait).argmax(1)
    s["tokens"] = torch.roll(tokens, 1).int()
    s["uniforms"] = torch.rand(rows, device="cuda", generator=g)
    s["next_tokens"] = torch.empty(rows, dtype=torch.int32, device="cuda")
    s["accepted"] = torch.empty(case["batch"], dtype=torch.int32, device="cuda")
    return s


# ----------------------------------------------------------------- plain forms
def _turn(x, s):
    """Rows x [T][H][D] in 32 bits, turned."""
    case = s["case"]
    first, rot = case["first"], case["rot"]
    angle = s["positions"].double().T[:, s["axis"]] * s["frequency"]   # 64 bits: positions are far
    cos, sin = torch.cos(angle).float()[:, None], torch.sin(angle).float()[:, None]
    x = x.float()
    part = x[..., first:first + rot]
    if case["pairs"] == "halves":
        a, b = part.chunk(2, -1)
        part = torch.cat([a * cos - b * sin, b * cos + a * sin], -1)
    else:
        a, b = part[..., 0::2], part[..., 1::2]
        part = torch.stack([a * cos - b * sin, b * cos + a * sin], -1).flatten(-2)
    return torch.cat([x[..., :first], part, x[..., first + rot:]], -1)


def _plain_rotary(s):
    case = s["case"]
    s["q_out"] = _turn(s["q"], s).bfloat16()
    if case["op"] == "embed":
        return s["q_out"]
    there = s["slots"] >= 0
    page, off = s["slots"][there] // case["page"], s["slots"][there] % case["page"]
    k = _turn(s["k_new"], s)
    _plain_append(s, "k", k[there], page, off)
    if _has_v(case):
        _plain_append(s, "v", s["v_new"].float()[there], page, off)
    return _rotary_outputs(s)


def _plain_append(s, x, rows, page, off):
    gran = s["case"]["gran"]
    if gran == "token":
        scale = rows.abs().amax(2) / 448
        s[x + "_scales"][page, :, off] = scale
    else:
        scale = s[x + "_scales"][None]
    scale = scale[..., None]
    codes = (torch.where(scale > 0, rows / scale, 0)).clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)
    s[x + "_cache"][page, :, off] = codes


def _rotary_outputs(s):
    got = {"q": s["q_out"]}
    for x in "kv" if _has_v(s["case"]) else "k":
        got[x] = s[x + "_cache"].view(torch.float8_e4m3fn)
        got[x + "_scales"] = s[x + "_scales"]
    return got


def _plain_copy(s):
    src, dst = s["pairs"].long().T
    for x in _arrays(s):
        x[:, dst] = x[:, src]
    return _copy_outputs(s)


def _arrays(s):
    return [s[x] for x in ("k_cache", "v_cache", "k_scales", "v_scales") if x in s]


def _copy_outputs(s):
    return [x.view(torch.float8_e4m3fn) if x.dtype == torch.uint8 else x for x in _arrays(s)]


def _plain_verify(s):
    p, q, u, start = s["target"], s["draft"], s["uniforms"], s["q_start"].long()
    rows, vocab = p.shape
    n = start.diff()
    request = torch.repeat_interleave(torch.arange(len(n), device="cuda"), n, output_size=rows)
    place = torch.arange(rows, device="cuda") - start[request]
    drafted = place < n[request] - 1                          # a drafted token follows this row
    token = torch.roll(s["tokens"].long(), -1)
    at = torch.arange(rows, device="cuda")
    px = p[at, token].double()
    qx = q[at, token].double() if q is not None else 1.0
    fine = drafted & (u.double() * qx < px)                   # the product is exact in 64 bits
    # accepted: the rows before a request's first that is not fine
    place_bad = torch.where(fine, n[request], place)
    accepted = torch.full_like(n, rows).scatter_reduce(0, request, place_bad, "amin")
    last = start[:-1] + accepted                              # the row whose next token is drawn
    rejected = accepted < n - 1
    weight = p[last].float()
    if q is not None:
        other = torch.where(rejected[:, None], q[last].float(), 0)
    else:
        other = torch.zeros_like(weight)
        other[torch.arange(len(n), device="cuda"), token[last]] = rejected.float()
    weight = (weight - other).clamp(0, 1)
    whole = (weight.double() * 2.0 ** WEIGHT_BITS).floor().long()
    total = whole.cumsum(1)
    uniform = (u[start[1:] - 1].double() * 2.0 ** UNIFORM_BITS).floor().long()
    all_of = total[:, -1]
    # floor(all_of * uniform / 2^24), in two halves of all_of
    threshold = ((all_of >> 32) * uniform << (32 - UNIFORM_BITS)) + ((all_of & 0xFFFFFFFF) * uniform >> UNIFORM_BITS)
    drawn = (total <= threshold[:, None]).sum(1)
    out = torch.where(place < accepted[request], token, -1)
    out[last] = drawn
    return {"next": out.int(), "accepted": accepted.int()}


# ------------------------------------------------------------------------ run
def run(state):
    s = state
    case = s["case"]
    op = case["op"]
    if not own:
        return {"rotary": _plain_rotary, "embed": _plain_rotary, "copy": _plain_copy, "verify": _plain_verify}[op](s)
    import paged_fp8_kv_02_gb300 as pf
    if op in ("rotary", "embed"):
        if "rotary" not in s:   # the model's frequencies, laid out once
            s["rotary"] = pf.Rotary(s["frequencies"], axes=s["axes"], first=case["first"], neighbours=case["pairs"] == "neighbours")
        if op == "embed":
            pf.rotary_embed(s["q_out"], s["q"], s["positions"], s["rotary"])
            return s["q_out"]
        gran = {"tensor": pf.SCALE_TENSOR, "head": pf.SCALE_HEAD, "token": pf.SCALE_TOKEN}[case["gran"]]
        pf.rotary_append_fp8(s["q_out"], s["q"], s["k_new"], s.get("v_new"), s["k_cache"], s.get("v_cache"), s["slots"],
                             s["positions"], s["rotary"], gran, s["k_scales"], s.get("v_scales"))
        return _rotary_outputs(s)
    if op == "copy":
        if "arrays" not in s:   # the caches of all layers, listed once
            s["arrays"] = pf.PagedArrays([layer for x in _arrays(s) for layer in x])
        pf.copy_pages(s["arrays"], s["pairs"])
        return _copy_outputs(s)
    pf.verify_drafts(s["next_tokens"], s["accepted"], s["target"], s["draft"], s["tokens"], s["uniforms"], s["q_start"])
    return {"next": s["next_tokens"], "accepted": s["accepted"]}


# ---------------------------------------------------------- values in 64 bits
def _code_values():
    """The 256 values of the format in double: sign, 4 exponent bits of bias 7,
    3 mantissa bits, subnormals, no infinity."""
    c = np.arange(256)
    e, m = (c >> 3) & 15, c & 7
    v = np.where(e == 0, m * 2.0 ** -9, (8 + m) * 2.0 ** (e - 10.0))
    v[(c & 127) == 127] = np.nan
    return torch.from_numpy(np.where(c & 128, -v, v)).cuda()


def _nearest_value(x):
    """Nearest e4m3 value of doubles, ties to even, saturating."""
    e = torch.floor(torch.log2(x.abs().clamp(min=2.0 ** -6)))
    step = torch.exp2(e - 3)
    return (torch.round(x / step) * step).clamp(-448, 448)


def _turned(x, s):
    """Rows x in 64 bits, each pair as a complex number times e^(i angle)."""
    case = s["case"]
    half, first = case["rot"] // 2, case["first"]
    i = torch.arange(half, device="cuda")
    if case["pairs"] == "halves":
        real, imag = first + i, first + half + i
    else:
        real, imag = first + 2 * i, first + 2 * i + 1
    angle = torch.stack([s["positions"][a].double() * f for a, f in zip(s["axes"].tolist(), s["frequencies"].tolist())], 1)
    x = x.double()
    z = torch.complex(x[..., real], x[..., imag]) * torch.polar(torch.ones_like(angle), angle)[:, None]
    x[..., real], x[..., imag] = z.real, z.imag
    return x


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "copy":
        came_from = torch.arange(case["pages"], device="cuda")
        for src, dst in s["pairs"].tolist():
            came_from[dst] = src
        value = _code_values()
        return [(value[x.long()] if x.dtype == torch.uint8 else x.double()).index_select(1, came_from) for x in _arrays(s)]
    if op == "embed":
        return _turned(s["q"], s)
    if op == "rotary":
        got = {"q": _turned(s["q"], s)}
        there = torch.nonzero(s["slots"] >= 0)[:, 0]
        page, off = s["slots"][there] // case["page"], s["slots"][there] % case["page"]
        for x in "kv" if _has_v(case) else "k":
            rows = (_turned(s["k_new"], s) if x == "k" else s["v_new"].double())[there]
            cache, scales = _code_values()[s[x + "_cache"].long()], s[x + "_scales"].double()
            if case["gran"] == "token":
                scale = rows.abs().amax(2) / 448
                scales[page, :, off] = scale
            else:
                scale = scales.expand(1, case["hkv"])
            cache[page, :, off] = _nearest_value(torch.nan_to_num(rows / scale[..., None]))
            got[x], got[x + "_scales"] = cache, scales
        return got
    start, tokens, u = s["q_start"].tolist(), s["tokens"].tolist(), s["uniforms"].tolist()
    following, accepted = [-1] * len(tokens), []
    for lo, hi in zip(start, start[1:]):
        kept = 0
        while kept < hi - lo - 1:
            x = tokens[lo + kept + 1]
            qx = 1.0 if s["draft"] is None else float(s["draft"][lo + kept, x])
            if not u[lo + kept] * qx < float(s["target"][lo + kept, x]):
                break
            following[lo + kept] = x
            kept += 1
        accepted.append(kept)
        weight = s["target"][lo + kept].float().cpu().numpy()
        if kept < hi - lo - 1:
            if s["draft"] is not None:
                weight = weight - s["draft"][lo + kept].float().cpu().numpy()
            else:
                weight[tokens[lo + kept + 1]] -= np.float32(1)
        whole = np.floor(np.clip(weight, 0, 1).astype(np.float64) * 2.0 ** WEIGHT_BITS).astype(np.int64)
        total = np.cumsum(whole)
        bar = int(total[-1]) * int(u[hi - 1] * 2 ** UNIFORM_BITS) >> UNIFORM_BITS
        following[lo + kept] = int(np.searchsorted(total, bar, side="right"))
    return {"next": torch.tensor(following, dtype=torch.int32), "accepted": torch.tensor(accepted, dtype=torch.int32)}
