"""Cases, plain forms and exact values of the block-scaled and block-sparse
operators of the paged e4m3 cache.

Five operators, named by a case's "op":

  append   kv_append_fp8_block: new K/V rows into pages that hold one scale
           per (page, KV head)
  decode   paged_decode_attn_scaled with those scales (SCALE_BLOCK)
  bounds   page_key_bounds: channelwise bounds of each page's keys in int8
  select   select_pages: the pages a query attends, by a score from the bounds
  sparse   paged_sparse_decode_attn: attention over the selected pages

A case gives its lengths as a geometric row from min_len to max_len over the
batch, so they are ragged and odd and known without a seed.  `own` is set from
outside: False runs the plain forms below, True the library's entry points.
"""
import math

import numpy as np
import torch

own = False

HEAD_DIM = 128
MIN_SCALE = 2.0 ** -126   # of a block of zeros
MIN_BOUND_SCALE = 2.0 ** -15


# ------------------------------------------------------------------ the cases
def listed():
    return [
        # one decode step of 64 requests: the smallest append, launch latency counts
        dict(name="append_step_b64", op="append", batch=64, hkv=8, page=16, min_len=256, max_len=1009, min_new=1, max_new=1),
        # prompts and chunks of 300 to 16,000 tokens, some after an earlier chunk
        dict(name="append_prompts_b8", op="append", batch=8, hkv=8, page=64, min_len=1021, max_len=17011, min_new=307, max_new=16001),
        # four short requests, 8/2 heads, 16-token pages
        dict(name="decode_tiny_b4", op="decode", batch=4, hq=8, hkv=2, page=16, min_len=16, max_len=300),
        # a decode step over long contexts: the largest call
        dict(name="decode_long_b8", op="decode", batch=8, hq=64, hkv=8, page=64, min_len=32771, max_len=262139),
        # bounds of the one page each of 64 requests has just appended to
        dict(name="bounds_step_b64", op="bounds", batch=64, hkv=8, page=16, min_len=256, max_len=4093, min_new=1, max_new=1),
        # bounds of whole prompts of 32K to 256K tokens
        dict(name="bounds_prompts_b4", op="bounds", batch=4, hkv=8, page=64, min_len=32771, max_len=262139, min_new=32771, max_new=262139),
        # one request of 128K tokens
        dict(name="select_b1_128k", op="select", batch=1, hq=64, hkv=8, page=64, min_len=131071, max_len=131071, top=64, sink=1, recent=2, block=True),
        # the ordinary batch: 64 requests of 256 to 32K tokens, 16-token pages
        dict(name="select_b64_32k", op="select", batch=64, hq=64, hkv=8, page=16, min_len=256, max_len=32768, top=128, sink=1, recent=2, block=False),
        # 8 requests of 256K to 1M tokens
        dict(name="select_b8_1m", op="select", batch=8, hq=64, hkv=8, page=64, min_len=262147, max_len=1048573, top=256, sink=1, recent=2, block=True),
        # one request: latency
        dict(name="sparse_b1_k64", op="sparse", batch=1, hq=64, hkv=8, page=64, min_len=131071, max_len=131071, top=64, gran="block"),
        # 64 requests, 16-token pages, lists of up to 128 pages
        dict(name="sparse_b64_k128", op="sparse", batch=64, hq=64, hkv=8, page=16, min_len=256, max_len=32768, top=128, gran="head"),
        # 8 long requests, 16K tokens each
        dict(name="sparse_b8_k256", op="sparse", batch=8, hq=64, hkv=8, page=64, min_len=32771, max_len=262139, top=256, gran="block"),
    ]


HEADS = [(8, 2), (64, 8), (48, 48), (16, 1), (20, 4), (32, 8), (7, 1), (12, 6)]
PAGES = [16, 32, 48, 64, 96, 128]


def _log_uniform(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    """A case of the ranges above: lengths from one token, every head layout
    and page size the library's tests use, batches of 1 to 96."""
    op = rng.choice(["append", "decode", "bounds", "select", "sparse"])
    hq, hkv = rng.choice(HEADS)
    page = rng.choice(PAGES)
    batch = _log_uniform(rng, 1, 96)
    # (token, head) rows of all requests together, padded to the longest
    room = {"append": 1 << 19, "decode": 1 << 23, "bounds": 1 << 22, "select": 1 << 25, "sparse": 1 << 23}[op]
    top_len = {"append": 16384, "decode": 262144, "bounds": 262144, "select": 1048576, "sparse": 262144}[op]
    longest = max(1, min(top_len, room // (batch * hkv)))
    # a choice of pages says something where there are many
    max_len = _log_uniform(rng, min(40 * page, longest) if op == "select" else 1, longest)
    case = dict(op=op, batch=batch, hkv=hkv, page=page, min_len=_log_uniform(rng, 1, max_len), max_len=max_len)
    if op in ("append", "bounds"):
        # a step, or a part, or the whole of every context
        kind = rng.choice(["step", "part", "whole"])
        lo, hi = case["min_len"], case["max_len"]
        if kind == "step":
            lo = hi = 1
        elif kind == "part":
            lo = _log_uniform(rng, 1, lo)
            hi = _log_uniform(rng, lo, hi)
        case.update(min_new=lo, max_new=hi)
    else:
        case["hq"] = hq
    npages = -(-max_len // page)
    if op in ("select", "sparse"):
        most = max(4, min(npages // 2, 65536 // page, 1024))
        case["top"] = _log_uniform(rng, 4 if op == "select" else 1, most)
    if op == "select":
        case["recent"] = rng.randint(0, min(3, case["top"] // 2))
        case["sink"] = rng.randint(0, min(2, case["top"] // 2 - case["recent"]))
        case["block"] = rng.random() < 0.5
    if op == "sparse":
        case["gran"] = rng.choice(["tensor", "head", "block"])
    return case


def _row(lo, hi, n):
    """n whole numbers, a geometric row from lo to hi (hi alone for n = 1)."""
    if n == 1:
        return [hi]
    return [int(round(lo * (hi / lo) ** (i / (n - 1)))) for i in range(n)]


def _lens(case):
    return _row(case["min_len"], case["max_len"], case["batch"])


def _new(case):
    # the longest new part on the shortest context where it fits
    return [min(n, m) for n, m in zip(_row(case["max_new"], case["min_new"], case["batch"])
                                      if case["min_new"] != case["max_new"] else [case["max_new"]] * case["batch"], _lens(case))]


def _touched(case):
    """Pages that hold at least one new token, over all requests."""
    p = case["page"]
    return sum((m - 1) // p - (m - n) // p + 1 for n, m in zip(_new(case), _lens(case)))


def work(case):
    op, hkv, p, d = case["op"], case["hkv"], case["page"], HEAD_DIM
    lens = _lens(case)
    pages = sum(-(-m // p) for m in lens)
    if op == "append":
        rows = sum(_new(case)) * hkv
        # K and V: bf16 rows read, codes written, one scale written per page and head
        return {"bytes": 2 * (rows * d * 3 + _touched(case) * hkv * 4), "flops": 2 * rows * d}
    if op == "bounds":
        # rows of the pages touched, up to the context's end
        rows = sum(m - (m - n) // p * p for n, m in zip(_new(case), lens)) * hkv
        return {"bytes": rows * d + _touched(case) * hkv * (2 * d + 4), "flops": 2 * rows * d}
    g = case["hq"] // hkv
    qo = case["batch"] * case["hq"] * d * 2
    if op == "decode":
        rows = sum(lens) * hkv
        return {"bytes": rows * 2 * d + pages * hkv * 8 + 2 * qo + case["batch"] * case["hq"] * 4, "flops": rows * 4 * d * g}
    if op == "select":
        # requests whose pages all fit the list need no scores
        scored = sum(n for n in (-(-m // p) for m in lens) if n > case["top"])
        return {"bytes": scored * hkv * (2 * d + 4 + (4 if case["block"] else 0)) + qo + case["batch"] * hkv * case["top"] * 4,
                "flops": scored * hkv * 4 * d}
    rows = sum(_listed_tokens(case)) * hkv
    return {"bytes": rows * 2 * d + case["batch"] * hkv * case["top"] * 4 + 2 * qo + case["batch"] * case["hq"] * 4,
            "flops": rows * 4 * d * g}


def _listed_tokens(case):
    """Tokens each (request, KV head) of a sparse case attends: the list holds
    the last page, which may be partial, and otherwise full ones."""
    p = case["page"]
    got = []
    for m in _lens(case):
        n = -(-m // p)
        got.append(m if n <= case["top"] else (case["top"] - 1) * p + (m - (n - 1) * p))
    return got


# --------------------------------------------------------------------- inputs
def _generator(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _tables(lens, page, rng, spare=3):
    """Block tables over a shuffled pool, -1 past each request's last page."""
    n = [-(-m // page) for m in lens]
    total = sum(n)
    ids = rng.permutation(total + spare).astype(np.int32)
    table = np.full((len(lens), max(n)), -1, np.int32)
    at = 0
    for b, k in enumerate(n):
        table[b, :k] = ids[at:at + k]
        at += k
    return torch.from_numpy(table).cuda(), total + spare


def _codes(shape, g):
    """e4m3 codes of rows as a quantiser leaves them: normal values whose
    largest in a block come near 448, a few channels larger than the others."""
    out = torch.empty(shape, dtype=torch.uint8, device="cuda")
    flat = out.view(-1, shape[-1])
    gain = torch.full((shape[-1],), 90.0, device="cuda")
    gain[torch.randint(0, shape[-1], (4,), device="cuda", generator=g)] = 160.0
    for part in flat.split(1 << 21):
        x = torch.randn(part.shape, device="cuda", generator=g)
        part.copy_((x * gain).clamp_(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8))
    return out


def _block_scales(pages, hkv, g):
    """Powers of two, as the append writes them."""
    return torch.exp2(torch.randint(-9, -5, (pages, hkv), device="cuda", generator=g).float())


def prepare(case, seed):
    g, rng = _generator(seed), np.random.default_rng(seed)
    op, hkv, page, lens = case["op"], case["hkv"], case["page"], _lens(case)
    table, pages = _tables(lens, page, rng)
    s = dict(case=case, block_tables=table, context_lens=torch.tensor(lens, dtype=torch.int32, device="cuda"))
    if op in ("append", "bounds"):
        new = _new(case)
        start = np.concatenate([[0], np.cumsum(new)]).astype(np.int32)
        s["new_start"] = torch.from_numpy(start).cuda()
        s["max_new_len"] = max(new)
    if op == "append":
        shape = (pages, hkv, page, HEAD_DIM)
        total = int(start[-1])
        for x in "kv":
            s[x + "_cache"] = _codes(shape, g)
            s[x + "_scales"] = _block_scales(pages, hkv, g)
            # rows whose size varies, so that some blocks' scales have to grow
            size = torch.exp2(torch.randn((total, 1, 1), device="cuda", generator=g))
            s[x + "_new"] = (torch.randn((total, hkv, HEAD_DIM), device="cuda", generator=g) * size).bfloat16()
        return s
    if op == "bounds":
        s["k_cache"] = _codes((pages, hkv, page, HEAD_DIM), g)
        s["bounds"] = torch.zeros((pages, hkv, 2, HEAD_DIM), dtype=torch.int8, device="cuda")
        s["bound_scales"] = torch.zeros((pages, hkv), device="cuda")
        return s
    s["q"] = torch.randn((case["batch"], case["hq"], HEAD_DIM), device="cuda", generator=g).bfloat16()
    s["softmax_scale"] = HEAD_DIM ** -0.5
    if op == "select":
        # lower and upper bounds around a channel's centre, as keys with a
        # common offset and some spread within a page give them
        centre = torch.randn((pages, hkv, HEAD_DIM), device="cuda", generator=g) * 25
        half = torch.rand((pages, hkv, HEAD_DIM), device="cuda", generator=g) * 50 + 8
        s["bounds"] = torch.stack([(centre - half).clamp_(-127, 127).floor_(), (centre + half).clamp_(-127, 127).ceil_()], 2).to(torch.int8)
        del centre, half
        s["bound_scales"] = torch.exp2(torch.randint(1, 3, (pages, hkv), device="cuda", generator=g).float())
        s["k_scales"] = _block_scales(pages, hkv, g) if case["block"] else None
        s["selected"] = torch.empty((case["batch"], hkv, case["top"]), dtype=torch.int32, device="cuda")
        return s
    shape = (pages, hkv, page, HEAD_DIM)
    s["k_cache"], s["v_cache"] = _codes(shape, g), _codes(shape, g)
    gran = case.get("gran", "block")
    for x in "kv":
        if gran == "block":
            s[x + "_scales"] = _block_scales(pages, hkv, g)
        else:
            s[x + "_scales"] = torch.rand(hkv if gran == "head" else 1, device="cuda", generator=g) * 0.02 + 0.005
    s["out"] = torch.empty_like(s["q"])
    s["lse"] = torch.empty((case["batch"], case["hq"]), device="cuda")
    if op == "sparse":
        chosen = np.full((case["batch"], hkv, case["top"]), -1, np.int32)
        for b, m in enumerate(lens):
            n = -(-m // page)
            k = min(n, case["top"])
            for h in range(hkv):  # distinct pages, the last one among them, in order
                chosen[b, h, :k] = np.sort(np.append(rng.choice(n - 1, k - 1, replace=False), n - 1))
        s["selected"] = torch.from_numpy(chosen).cuda()
    return s


# ----------------------------------------------------------------- plain forms
def _values(codes):
    return codes.view(torch.float8_e4m3fn).float()


def _e4m3(x):
    """Nearest e4m3 value's code, ties to even; |x| <= 448."""
    return x.to(torch.float8_e4m3fn).view(torch.uint8)


def _touched_pages(s):
    """For every page with a new token: its request, logical index and physical
    id, and the first new and the last attended row in it."""
    page = s["case"]["page"]
    m = s["context_lens"].long()
    n = s["new_start"].long().diff()
    most = (s["max_new_len"] + page - 1) // page + 1
    logical = ((m - n) // page)[:, None] + torch.arange(most, device="cuda")
    b, i = torch.nonzero(logical * page < m[:, None], as_tuple=True)
    logical = logical[b, i]
    first = (m[b] - n[b] - logical * page).clamp(min=0)
    end = (m[b] - logical * page).clamp(max=page)
    return b, logical, s["block_tables"][b, logical].long(), first, end


def _plain_append(s):
    page = s["case"]["page"]
    b, logical, phys, first, end = _touched_pages(s)
    row = torch.arange(page, device="cuda")
    is_new = (row >= first[:, None]) & (row < end[:, None])                         # [N][P]
    start, m = s["new_start"].long(), s["context_lens"].long()
    n = start.diff()
    token = (start[b] - (m[b] - n[b]) + logical * page)[:, None] + row              # row's index among the new ones
    token = torch.where(is_new, token, 0)
    for x in "kv":
        new = s[x + "_new"].float()[token].transpose(1, 2)                          # [N][H][P][D]
        mask = is_new[:, None, :, None]
        amax = torch.where(mask, new.abs(), 0).amax((2, 3))                         # [N][H]
        need = torch.exp2(torch.where(amax > 0, _shift_to(amax.double(), 448).clamp(min=-126), -126).float())
        has_old = (first > 0)[:, None]
        old = torch.where(has_old, s[x + "_scales"][phys], MIN_SCALE)
        scale = torch.maximum(old, need)
        codes = s[x + "_cache"][phys]
        kept = _e4m3(_values(codes) * (old / scale)[:, :, None, None])
        kept = torch.where((row < first[:, None])[:, None, :, None], kept, codes)
        s[x + "_cache"][phys] = torch.where(mask, _e4m3((new / scale[:, :, None, None]).clamp(-448, 448)), kept)
        s[x + "_scales"][phys] = scale
    return _append_outputs(s)


def _append_outputs(s):
    return {"k": s["k_cache"].view(torch.float8_e4m3fn), "v": s["v_cache"].view(torch.float8_e4m3fn),
            "k_scales": s["k_scales"], "v_scales": s["v_scales"]}


def _plain_bounds(s):
    page = s["case"]["page"]
    _, _, phys, _, end = _touched_pages(s)
    attended = (torch.arange(page, device="cuda") < end[:, None])[:, None, :, None]
    x = _values(s["k_cache"][phys])
    lo = torch.where(attended, x, torch.inf).amin(2)
    hi = torch.where(attended, x, -torch.inf).amax(2)
    amax = torch.maximum(lo.abs(), hi.abs()).amax(2)
    scale = torch.exp2(_shift_to(amax.double(), 127)).clamp(min=MIN_BOUND_SCALE).float()
    s["bounds"][phys] = torch.stack([torch.floor(lo / scale[..., None]), torch.ceil(hi / scale[..., None])], 2).to(torch.int8)
    s["bound_scales"][phys] = scale
    return {"bounds": s["bounds"], "scales": s["bound_scales"]}


def _shift_to(x, most):
    """The smallest whole e with x <= most * 2^e."""
    mantissa, exponent = torch.frexp(x / most)
    return exponent - (mantissa == 0.5).int()


def _group_query(q, hkv):
    """The positive and the negative part of a group's queries, summed over
    its heads, in 8-bit whole numbers -> [B][Hkv][2][D] (negative part first)."""
    b, hq, d = q.shape
    q = q.float().view(b, hkv, hq // hkv, d)
    exponent = torch.frexp(q.abs().amax((2, 3), keepdim=True))[1]
    whole = torch.round(torch.ldexp(q, 14 - exponent))
    parts = torch.stack([whole.clamp(max=0).sum(2), whole.clamp(min=0).sum(2)], 2)
    most = parts.abs().amax((2, 3), keepdim=True)
    shift = _shift_to(most.double(), 127).clamp(min=0).float()
    return torch.round(parts * torch.exp2(-shift))


def _plain_select(s):
    case = s["case"]
    page, top = case["page"], case["top"]
    table = s["block_tables"].long()
    npages = (s["context_lens"].long() + page - 1) // page
    phys = table.clamp(min=0)
    query = _group_query(s["q"], case["hkv"])
    score = torch.einsum("bnhcd,bhcd->bhn", s["bounds"][phys].float(), query)      # whole numbers below 2^24: exact
    scale = s["bound_scales"][phys] * (s["k_scales"][phys] if case["block"] else 1.0)
    score = score * scale.transpose(1, 2)
    index = torch.arange(table.shape[1], device="cuda")
    there = index < npages[:, None]
    always = there & ((index < case["sink"]) | (index >= npages[:, None] - case["recent"]))
    score = torch.where(always[:, None], torch.inf, torch.where(there[:, None], score, -torch.inf))
    order = torch.sort(score, dim=2, descending=True, stable=True)[1][:, :, :top]
    count = npages.clamp(max=top)[:, None, None]
    far = table.shape[1]
    slot = torch.arange(order.shape[2], device="cuda")
    chosen = torch.sort(torch.where(slot < count, order, far), dim=2)[0]
    s["selected"].fill_(-1)
    s["selected"][:, :, :order.shape[2]] = torch.where(chosen < far, chosen, -1).int()
    return s["selected"]


def _attend(q, k, v, there):
    """Softmax attention of q [B][H][G][D] over k, v [B][H][T][D] where `there`
    [B][H][T] is set -> output and log-sum-exp."""
    score = torch.einsum("bhgd,bhtd->bhgt", q, k)
    score = torch.where(there[:, :, None], score, -torch.inf)
    m = score.amax(3, keepdim=True)
    p = torch.exp(score - m)
    total = p.sum(3, keepdim=True)
    out = torch.einsum("bhgt,bhtd->bhgd", p / total, v)
    return out.flatten(1, 2).bfloat16(), (m + torch.log(total)).flatten(1)


def _scale_of(s, x, phys, head):
    """Scale of the pages `phys` at the heads `head`, by granularity."""
    gran, scales = s["case"].get("gran", "block"), s[x + "_scales"]
    return scales[phys, head] if gran == "block" else (scales[head] if gran == "head" else scales[0]).expand(phys.shape)


def _plain_attention(s):
    case = s["case"]
    b, hkv, page = case["batch"], case["hkv"], case["page"]
    npages = (s["context_lens"].long() + page - 1) // page
    if case["op"] == "sparse":
        logical = s["selected"].long()
    else:
        index = torch.arange(s["block_tables"].shape[1], device="cuda")
        logical = torch.where(index < npages[:, None], index, -1)[:, None].expand(b, hkv, -1)
    at = logical.clamp(min=0)
    phys = torch.gather(s["block_tables"].long()[:, None].expand(b, hkv, -1), 2, at).clamp(min=0)
    head = torch.arange(hkv, device="cuda")[:, None]
    token = logical[..., None] * page + torch.arange(page, device="cuda")
    there = (logical[..., None] >= 0) & (token < s["context_lens"].long()[:, None, None, None])
    k = (_values(s["k_cache"][phys, head]) * _scale_of(s, "k", phys, head)[..., None, None]).flatten(2, 3)
    v = (_values(s["v_cache"][phys, head]) * _scale_of(s, "v", phys, head)[..., None, None]).flatten(2, 3)
    q = s["q"].float().view(b, hkv, -1, HEAD_DIM) * s["softmax_scale"]
    out, lse = _attend(q, k, v, there.flatten(2))
    return {"out": out, "lse": lse}


# ------------------------------------------------------------------------ run
def run(state):
    s = state
    op = s["case"]["op"]
    if not own:
        return {"append": _plain_append, "bounds": _plain_bounds, "select": _plain_select,
                "decode": _plain_attention, "sparse": _plain_attention}[op](s)
    import paged_fp8_kv_02_gb300 as pf
    if op == "append":
        pf.kv_append_fp8_block(s["k_new"], s["v_new"], s["k_cache"], s["v_cache"], s["k_scales"], s["v_scales"],
                               s["block_tables"], s["context_lens"], s["new_start"], s["max_new_len"])
        return _append_outputs(s)
    if op == "bounds":
        pf.page_key_bounds(s["bounds"], s["bound_scales"], s["k_cache"], s["block_tables"], s["context_lens"],
                           s["new_start"], s["max_new_len"])
        return {"bounds": s["bounds"], "scales": s["bound_scales"]}
    if op == "select":
        c = s["case"]
        pf.select_pages(s["selected"], s["q"], s["bounds"], s["bound_scales"], s["block_tables"], s["context_lens"],
                        c["page"], sink_pages=c["sink"], recent_pages=c["recent"], k_scales=s["k_scales"])
        return s["selected"]
    if op == "decode":  # the call allocates a workspace where it is given none; the program keeps it
        s["workspace"] = pf.paged_decode_attn_scaled(
            s["out"], s["q"], s["k_cache"], s["v_cache"], pf.SCALE_BLOCK, s["k_scales"], s["v_scales"],
            s["block_tables"], s["context_lens"], s["softmax_scale"], workspace=s.get("workspace"), lse_out=s["lse"])
    else:
        gran = {"tensor": pf.SCALE_TENSOR, "head": pf.SCALE_HEAD, "block": pf.SCALE_BLOCK}[s["case"]["gran"]]
        pf.paged_sparse_decode_attn(s["out"], s["q"], s["k_cache"], s["v_cache"], gran, s["k_scales"], s["v_scales"],
                                    s["selected"], s["block_tables"], s["context_lens"], s["softmax_scale"],
                                    lse_out=s["lse"])
    return {"out": s["out"], "lse": s["lse"]}


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


def _power_of_two_over(x, least):
    """The smallest power of two that is at least x, and at least `least`.  The
    values here are multiples of 2^-8 of a power of two over 448 or 127, so a
    hair off the logarithm takes no step too many and none too few."""
    return torch.exp2(torch.ceil(torch.log2(x) - 1e-9)).clamp(min=least)


def exact(case, seed):
    s = prepare(case, seed)
    op, hkv, page, lens = case["op"], case["hkv"], case["page"], _lens(case)
    value = _code_values()
    table = s["block_tables"].long()
    if op in ("append", "bounds"):
        new = _new(case)
        start = s["new_start"].tolist()
    if op == "append":
        got = {}
        for x in "kv":
            cache = value[s[x + "_cache"].long()]
            scales = s[x + "_scales"].double()
            rows = s[x + "_new"].double()
            for b in range(case["batch"]):
                for i in range((lens[b] - new[b]) // page, (lens[b] - 1) // page + 1):
                    at = int(table[b, i])
                    lo, hi = max(0, lens[b] - new[b] - i * page), min(page, lens[b] - i * page)
                    t = start[b] + i * page + lo - (lens[b] - new[b])
                    block = rows[t:t + hi - lo].transpose(0, 1)                     # [H][rows][D]
                    need = _power_of_two_over(block.abs().amax((1, 2)) / 448, MIN_SCALE)
                    old = scales[at].clone()
                    if lo:
                        need = torch.maximum(need, old)
                        cache[at, :, :lo] = _nearest_value(cache[at, :, :lo] * (old / need)[:, None, None])
                    scales[at] = need
                    cache[at, :, lo:hi] = _nearest_value(block / need[:, None, None])
            got[x], got[x + "_scales"] = cache, scales
        return got
    if op == "bounds":
        scales = s["bound_scales"].double()
        for b in range(case["batch"]):
            first, last = (lens[b] - new[b]) // page, (lens[b] - 1) // page
            for lo in range(first, last + 1, 256):
                ids = table[b, lo:min(lo + 256, last + 1)]
                x = value[s["k_cache"][ids].long()].abs()
                tokens = torch.arange(lo, lo + len(ids), device="cuda")[:, None] * page + torch.arange(page, device="cuda")
                x[(tokens >= lens[b])[:, None].expand(-1, hkv, -1)] = 0
                a = x.amax((2, 3))
                scales[ids] = _power_of_two_over(a / 127, MIN_BOUND_SCALE)
        return {"bounds": None, "scales": scales}
    if op == "select":
        return None
    out = torch.zeros((case["batch"], case["hq"], HEAD_DIM), dtype=torch.float64, device="cuda")
    lse = torch.full((case["batch"], case["hq"]), -torch.inf, dtype=torch.float64, device="cuda")
    group, gran = case["hq"] // hkv, case.get("gran", "block")
    for b in range(case["batch"]):
        for h in range(hkv):
            logical = torch.arange(-(-lens[b] // page), device="cuda")
            if op == "sparse":
                logical = s["selected"][b, h].long()
                logical = logical[logical >= 0]
            ids = table[b, logical]
            token = (logical[:, None] * page + torch.arange(page, device="cuda")).flatten() < lens[b]
            kv = []
            for x in "kv":
                scale = s[x + "_scales"].double()
                scale = scale[ids, h][:, None, None] if gran == "block" else scale[h if gran == "head" else 0]
                kv.append((value[s[x + "_cache"][ids, h].long()] * scale).flatten(0, 1)[token])
            heads = slice(h * group, (h + 1) * group)
            score = s["q"][b, heads].double() @ kv[0].T * s["softmax_scale"]
            lse[b, heads] = torch.logsumexp(score, 1)
            out[b, heads] = torch.softmax(score, 1) @ kv[1]
    return {"out": out, "lse": lse}
