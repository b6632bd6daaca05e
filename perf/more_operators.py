"""The operators on a round's key/value cache, as measured cases.

A round of speculative decoding feeds gamma+1 tokens of each sequence through
the target and keeps what the verify step accepts.  Three operators work on
the paged cache that those tokens are written to and attended from:

``plan``    the bookkeeping between two rounds, on the GPU: lengths move by the
            tokens that the last round kept, pages that it no longer needs go
            back to the free list, the next round's pages come from it, and
            every row gets its slot and position.
``store``   a round's (or a prompt's) keys and values quantised to 4 bits into
            their slots, and read back from them.
``attend``  the attention of a round's gamma+1 rows over the 4-bit pages: row i
            of sequence b sees the cached positions 0 .. lengths[b] + i.

The cache is one uint8 tensor [pages, heads, page * (D + 8)].  A head's block
of a page holds, one after another: the codes of its keys (page rows of D / 2
bytes, channel 2j in the low half of byte j), the codes of its values (the
rows of two neighbouring tokens interleaved by units of four channels: unit j
of the even token, unit j of the odd one, unit j+1 ...), and for every token
four numbers of the model's type: scale and offset of its key, scale and
offset of its value.  A held value is scale * code + offset.

``run`` computes an operator's plain form from elementary torch operations in
32 bits where ``own`` is false, and calls the package where it is true;
``exact`` computes the definition in 64 bits.
"""

import math

import torch

own = False

_TYPES = {"bf16": torch.bfloat16, "f16": torch.float16}
# a drawn case's work stays below the largest listed case's of its kind
_MOST = {"store": 6.0e7, "attend": 1.0e9}


def _package():
    import speculative_decoding_verification_46_gb300 as package

    return package


def _plan(name, B, gamma, page, length, ragged):
    """length: most tokens that a sequence has cached; ragged: tokens differ by
    sequence, some sequences take no part in the round."""
    return {"name": name, "op": "plan", "B": B, "gamma": gamma, "page": page, "length": length, "ragged": ragged}


def _store(name, B, gamma, heads, D, page, dtype, fused):
    """fused: keys and values are slices of the projections' common output;
    half of the rows of a sequence are then padding."""
    return {"name": name, "op": "store", "B": B, "gamma": gamma, "heads": heads, "D": D, "page": page, "dtype": dtype, "fused": fused}


def _attend(name, B, gamma, heads, group, D, page, length, dtype, ragged, lse):
    """group: query heads that share a key/value head; length: most tokens that
    a sequence has cached (the others have at least half); lse: the logarithm
    of each row's sum is wanted too."""
    return {"name": name, "op": "attend", "B": B, "gamma": gamma, "heads": heads, "group": group, "D": D, "page": page, "length": length,
            "dtype": dtype, "ragged": ragged, "lse": lse}


def listed():
    return [
        # one request's next round: all latency
        _plan("plan_b1_g4_page16", 1, 4, 16, 500, False),
        # a large batch between two rounds, drafts of different lengths
        _plan("plan_b1024_g8_page32_ragged", 1024, 8, 32, 4096, True),
        # prompts are admitted: a slot for every token of 64 prompts
        _plan("plan_b64_g4095_page16", 64, 4095, 16, 1, False),
        # one new token of one request: all latency
        _store("store_b1_g0_h8_d128_bf16", 1, 0, 8, 128, 16, "bf16", False),
        # prompts of odd length in half precision with small heads, out of the projections' common output
        _store("store_b9_g776_h5_d64_f16_fused", 9, 776, 5, 64, 16, "f16", True),
        # a long prompt's chunks
        _store("store_b8_g4095_h8_d128_bf16", 8, 4095, 8, 128, 64, "bf16", False),
        # one request, one new token, a short chat: all latency
        _attend("attend_b1_g0_h8x4_d128_len700_bf16", 1, 0, 8, 4, 128, 16, 700, "bf16", False, False),
        # a small batch in half precision with odd head counts and small heads, drafts of different lengths
        _attend("attend_b7_g3_h3x5_d64_len2500_f16_ragged", 7, 3, 3, 5, 64, 16, 2500, "f16", True, True),
        # decoding without drafts, a large batch
        _attend("attend_b128_g0_h8x8_d128_len4096_bf16", 128, 0, 8, 8, 128, 64, 4096, "bf16", False, False),
        # a verify round of a medium batch
        _attend("attend_b32_g4_h8x4_d128_len8192_bf16", 32, 4, 8, 4, 128, 64, 8192, "bf16", True, False),
        # a wide verify round with many query heads a key/value head
        _attend("attend_b48_g8_h4x8_d128_len6000_bf16", 48, 8, 4, 8, 128, 32, 6000, "bf16", False, False),
        # few requests with long documents: the largest
        _attend("attend_b4_g3_h8x4_d128_len240000_bf16", 4, 3, 8, 4, 128, 64, 240000, "bf16", False, True),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(max(lo, hi))))))


def draw(rng):
    op = rng.choice(["plan", "store", "attend", "attend"])
    page = rng.choice([16, 32, 64, 128])
    ragged = rng.random() < 0.5
    if op == "plan":
        prompts = rng.random() < 0.3
        B = _log_int(rng, 1, 64 if prompts else 1024)
        gamma = _log_int(rng, 16, 4095) if prompts else rng.randint(0, 8)
        return _plan("", B, gamma, page, 1 if prompts else _log_int(rng, 1, 4096), ragged)
    D, dtype = rng.choice([64, 128, 128]), rng.choice(["bf16", "bf16", "f16"])
    heads = rng.randint(1, 8)
    if op == "store":
        rows = _log_int(rng, 1, _MOST[op] / (heads * D) / 2)
        B = min(rows, _log_int(rng, 1, 64))
        return _store("", B, max(0, rows // B - 1), heads, D, page, dtype, ragged)
    group, gamma = rng.choice([1, 2, 3, 4, 5, 6, 8]), rng.randint(0, 8)
    B = _log_int(rng, 1, 128)
    most = _MOST[op] * min(1.0, 16 / (group * (gamma + 1)))
    length = _log_int(rng, 16, max(17, min(131072, most / (B * heads * D))))
    return _attend("", B, gamma, heads, group, D, page, length, dtype, ragged, rng.random() < 0.3)


# ------------------------------------------------------------------ inputs

def _ints(gen, lo, hi, shape):
    """Whole numbers lo .. hi, both included."""
    return torch.randint(lo, hi + 1, shape, generator=gen, device="cuda", dtype=torch.int32)


def _drafts(case, gen):
    """Drafts of each sequence this round; -1: it takes no part (the first one does)."""
    if not case["ragged"]:
        return None
    drafts = _ints(gen, -1, case["gamma"], (case["B"],))
    drafts[0] = case["gamma"]
    return drafts


def _pages_of(tokens, page):
    return (tokens + page - 1) // page


def _deal(need, width, gen, spare):
    """Pages in no order for sequences that need so many each: (table [B, width] with -1 behind, ids left over)."""
    total = int(need.sum())
    ids = torch.randperm(total + spare, generator=gen, device="cuda", dtype=torch.int32)
    at = torch.arange(width, device="cuda")
    first = need.cumsum(0) - need
    index = (first[:, None] + at).clamp(max=total + spare - 1)
    return torch.where(at < need[:, None], ids[index.long()], -1), ids[total:]


def _prepare_plan(case, gen):
    B, gamma, page, length = case["B"], case["gamma"], case["page"], case["length"]
    s = {"case": case}
    s["lengths"] = _ints(gen, length // 2, length, (B,))
    # two rounds: the first keeps some of the tokens before it, the second takes them back
    s["kept"] = _ints(gen, 0, min(gamma, 8) + 1, (B,))
    s["taken"] = -s["kept"]
    s["gamma_a"], s["gamma_b"] = _drafts(case, gen), _ints(gen, -1, min(gamma, 8), (B,))
    need = _pages_of(s["lengths"] + s["gamma_b"] + 1, page)
    width = -(-(length + 2 * gamma + 16) // page)
    most = B * (_pages_of(gamma + min(gamma, 8) + 2, page) + 1)      # pages that the first round may take at once
    s["table"], left = _deal(need, width, gen, most)
    s["blocks"] = need.to(torch.int32)
    s["free"] = torch.full((B * width + most,), -1, dtype=torch.int32, device="cuda")
    s["free"][:most] = left
    s["free_count"] = torch.tensor([most], dtype=torch.int32, device="cuda")
    return s


def _hold(x):
    """Codes, scale and offset of rows [.., D] (the format's definition, in 32 bits)."""
    f = x.float()
    lo = f.amin(-1, keepdim=True)
    scale = ((f.amax(-1, keepdim=True) - lo) / 15.0).to(x.dtype).float()
    inverse = torch.where(scale < 2.0 ** -126, 0.0, 1.0 / scale)
    codes = torch.round((f - lo) * inverse).clamp(0, 15).to(torch.uint8)
    return codes, scale.to(x.dtype), lo.to(x.dtype)


def _pack(codes):
    """Two channels a byte."""
    return codes[..., 0::2] | (codes[..., 1::2] << 4)


def _parts(cache, page, dtype):
    """Views of a cache: keys [p, H, page, D/2], values [p, H, page/2, D/4, 2, 2], numbers [p, H, page, 4]."""
    n, heads, size = cache.shape
    half = (size // page - 8) // 2
    keys = cache[..., :page * half].unflatten(-1, (page, half))
    values = cache[..., page * half:2 * page * half].unflatten(-1, (page // 2, half // 2, 2, 2))
    return keys, values, cache[..., 2 * page * half:].view(dtype).unflatten(-1, (page, 4))


def _model_rows(shape, gen, dtype, keys):
    """Keys (some channels far from zero, as rotary models have them) or values."""
    x = torch.randn(shape, generator=gen, device="cuda")
    if keys:
        x += 2.0 * torch.randn(shape[-1], generator=gen, device="cuda")
    return x.to(dtype)


def _prepare_store(case, gen):
    B, rows, heads, D, page = case["B"], case["gamma"] + 1, case["heads"], case["D"], case["page"]
    dtype = _TYPES[case["dtype"]]
    s = {"case": case}
    if case["fused"]:
        both = torch.empty(B, rows, 6 * heads, D, dtype=dtype, device="cuda")
        s["k"], s["v"] = both[:, :, 4 * heads:5 * heads], both[:, :, 5 * heads:]
        s["k"].copy_(_model_rows((B, rows, heads, D), gen, dtype, True))
        s["v"].copy_(_model_rows((B, rows, heads, D), gen, dtype, False))
    else:
        s["k"], s["v"] = _model_rows((B, rows, heads, D), gen, dtype, True), _model_rows((B, rows, heads, D), gen, dtype, False)
    start = _ints(gen, 0, 3 * page, (B,))
    used = _ints(gen, 1, rows, (B,)) if case["fused"] else torch.full((B,), rows, device="cuda")
    width = -(-(rows + 3 * page) // page)
    table, left = _deal(_pages_of(start + rows, page), width, gen, 1)
    at = torch.arange(rows, device="cuda")
    position = (start[:, None] + at).long()
    slots = table.gather(1, position // page) * page + position % page
    s["slots"] = torch.where(at < used[:, None], slots, -1).to(torch.int32)
    pages = int((table >= 0).sum()) + left.numel()
    s["cache"] = torch.zeros(pages, heads, page * (D + 8), dtype=torch.uint8, device="cuda")
    return s


def _prepare_attend(case, gen):
    B, rows, heads, D, page, length = case["B"], case["gamma"] + 1, case["heads"], case["D"], case["page"], case["length"]
    dtype = _TYPES[case["dtype"]]
    s = {"case": case}
    s["lengths"] = _ints(gen, length // 2, length, (B,))
    s["lengths"][0] = length
    s["gamma_b"] = _drafts(case, gen)
    s["table"], left = _deal(_pages_of(s["lengths"] + rows, page), -(-(length + rows) // page), gen, 3)
    pages = int((s["table"] >= 0).sum()) + left.numel()
    s["cache"] = torch.empty(pages, heads, page * (D + 8), dtype=torch.uint8, device="cuda")
    step = max(1, (1 << 27) // (heads * page * D))
    for p in range(0, pages, step):
        keys, values, numbers = _parts(s["cache"][p:p + step], page, dtype)
        shape = (keys.shape[0], heads, page, D)
        codes, numbers[..., 0:1], numbers[..., 1:2] = _hold(_model_rows(shape, gen, dtype, True))
        keys.copy_(_pack(codes))
        codes, numbers[..., 2:3], numbers[..., 3:4] = _hold(_model_rows(shape, gen, dtype, False))
        values.copy_(_pack(codes).unflatten(2, (page // 2, 2)).unflatten(-1, (D // 4, 2)).transpose(3, 4))
    s["q"] = (1.5 * torch.randn(B, rows, heads * case["group"], D, generator=gen, device="cuda")).to(dtype)
    return s


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    if case["op"] == "plan":
        return _prepare_plan(case, gen)
    return _prepare_store(case, gen) if case["op"] == "store" else _prepare_attend(case, gen)


# ------------------------------------------------------------------ the plain forms

def _plain_round(s, kept, gamma_b):
    """One round's bookkeeping: the state moves in place, (slots, positions, status) are new."""
    page, table, free = s["case"]["page"], s["table"], s["free"]
    B, width = table.shape
    rows = s["case"]["gamma"] + 1
    at, cell = torch.arange(rows, device=table.device), torch.arange(width, device=table.device)
    s["lengths"].add_(kept).clamp_(min=0)
    count = torch.full_like(kept, rows) if gamma_b is None else gamma_b.clamp(-1, rows - 1) + 1
    need = _pages_of(s["lengths"] + count, page)
    held = s["blocks"].clone()
    long_ = need > width
    need = torch.where(long_, held, need)
    out, grow = (held - need).clamp(min=0), (need - held).clamp(min=0)
    there = s["free_count"] + out.sum()
    none = (grow > 0) & (grow.cumsum(0) > there)
    grow = torch.where(none, 0, grow)
    # what is no longer needed goes to the top of the free list, the last page of the last sequence first
    leaving = (cell >= need[:, None]) & (cell < held[:, None])
    rank = leaving.flatten().cumsum(0).view(B, width) - 1
    dump = free.numel()
    place = torch.where(leaving, there - 1 - rank, dump)
    longer = torch.cat([free, free[:1]])
    longer.scatter_(0, place.flatten().long(), table.flatten())
    free.copy_(longer[:dump])
    table.masked_fill_(leaving, -1)
    # new pages come from its top, the first page of the first sequence first
    coming = (cell >= held[:, None]) & (cell < (held + grow)[:, None])
    rank = coming.flatten().cumsum(0).view(B, width) - 1
    table.copy_(torch.where(coming, free[(there - 1 - rank).clamp(0, dump - 1).long()], table))
    s["blocks"].copy_(held - out + grow)
    s["free_count"].copy_(there - grow.sum())
    status = none.to(torch.int32) + 2 * long_.to(torch.int32)
    position = s["lengths"][:, None] + at
    inside = at < count[:, None]
    page_of = table.gather(1, (position // page).clamp(max=width - 1).long())
    slots = torch.where(inside & (status == 0)[:, None], page_of * page + position % page, -1)
    return slots.to(torch.int32), torch.where(inside, position, 0).to(torch.int32), status


def _plain_store(s):
    cache, page, slots = s["cache"], s["case"]["page"], s["slots"].long().flatten()
    keys, values, numbers = _parts(cache, page, s["k"].dtype)
    # a row without a slot is written to (and read from) one more page behind the cache
    used = torch.where(slots < 0, cache.shape[0] * page, slots)
    p, t = used // page, used % page
    back = []
    for_keys, for_values = s["k"].flatten(0, 1), s["v"].flatten(0, 1)
    heads, D = for_keys.shape[-2:]
    spare = lambda part: torch.cat([part, part[:1]])  # noqa: E731
    codes, scale, offset = _hold(for_keys)
    more, more_numbers = spare(keys), spare(numbers)
    more[p, :, t] = _pack(codes)
    more_numbers[p, :, t, 0], more_numbers[p, :, t, 1] = scale[..., 0], offset[..., 0]
    keys.copy_(more[:-1])
    got = more[p, :, t]
    held = torch.stack([got & 15, got >> 4], -1).flatten(-2).float()
    back.append(held * more_numbers[p, :, t, 0].float()[..., None] + more_numbers[p, :, t, 1].float()[..., None])
    codes, scale, offset = _hold(for_values)
    more = spare(values)
    more[p, :, t // 2, :, t % 2] = _pack(codes).unflatten(-1, (D // 4, 2))
    more_numbers[p, :, t, 2], more_numbers[p, :, t, 3] = scale[..., 0], offset[..., 0]
    values.copy_(more[:-1])
    numbers.copy_(more_numbers[:-1])
    got = more[p, :, t // 2, :, t % 2].flatten(-2)
    held = torch.stack([got & 15, got >> 4], -1).flatten(-2).float()
    back.append(held * more_numbers[p, :, t, 2].float()[..., None] + more_numbers[p, :, t, 3].float()[..., None])
    shape = s["k"].shape
    none = (slots < 0)[:, None, None]
    return torch.where(none, 0.0, back[0]).to(s["k"].dtype).view(shape), torch.where(none, 0.0, back[1]).to(s["k"].dtype).view(shape)


def _plain_attend(s):
    case, table, q = s["case"], s["table"], s["q"]
    B, rows, _, D = q.shape
    heads, group, page = case["heads"], case["group"], case["page"]
    keys, values, numbers = _parts(s["cache"][table.clamp(min=0).long().flatten()], page, q.dtype)
    tokens = table.shape[1] * page

    def held(codes, which):
        x = torch.stack([codes & 15, codes >> 4], -1).flatten(-2).float()
        x = x * numbers[..., which, None].float() + numbers[..., which + 1, None].float()
        return x.unflatten(0, (B, -1)).transpose(1, 2).reshape(B, heads, tokens, D)

    k = held(keys, 0)
    query = q.float().view(B, rows, heads, group, D).transpose(1, 2).reshape(B, heads, rows * group, D)
    x = query @ k.transpose(-1, -2) / math.sqrt(D)
    del k
    at, row = torch.arange(tokens, device=q.device), torch.arange(rows * group, device=q.device) // group
    sees = at <= (s["lengths"][:, None, None] + row[:, None])
    sees &= (table >= 0).repeat_interleave(page, 1)[:, None]
    x = torch.where(sees[:, None], x, -math.inf)
    top = x.amax(-1, keepdim=True)
    x = torch.exp(x - torch.where(top > -math.inf, top, 0.0))
    total = x.sum(-1, keepdim=True)
    o = x @ held(values.transpose(3, 4).flatten(-2).flatten(2, 3), 2) / torch.where(total > 0, total, 1.0)
    lse = (total.log() + top).squeeze(-1)
    o = o.view(B, heads, rows, group, D).transpose(1, 2).reshape(q.shape)
    lse = lse.view(B, heads, rows, group).transpose(1, 2).reshape(q.shape[:3])
    if s["gamma_b"] is not None:
        behind = torch.arange(rows, device=q.device) > s["gamma_b"][:, None]
        o, lse = torch.where(behind[..., None, None], 0.0, o), torch.where(behind[..., None], 0.0, lse)
    return (o.to(q.dtype), lse) if case["lse"] else o.to(q.dtype)


def _round(s, kept, gamma_b):
    if not own:
        return _plain_round(s, kept, gamma_b)
    return _package().plan_round(s["lengths"], s["case"]["gamma"], s["case"]["page"], s["table"], s["blocks"], s["free"], s["free_count"],
                                 kept=kept, gamma_b=gamma_b)


def run(state):
    case = state["case"]
    if case["op"] == "plan":
        first = _round(state, state["kept"], state["gamma_a"])
        second = _round(state, state["taken"], state["gamma_b"])
        return first, second, state["lengths"], state["table"], state["blocks"], state["free"], state["free_count"]
    if case["op"] == "store":
        if not own:
            return _plain_store(state)
        _package().append_kv4(state["k"], state["v"], state["slots"], state["cache"])
        return _package().read_kv4(state["cache"], state["slots"], case["page"], state["k"].dtype)
    if not own:
        return _plain_attend(state)
    return _package().attend_kv4(state["q"], state["cache"], state["table"], state["lengths"], case["page"], gamma_b=state["gamma_b"],
                                 return_lse=case["lse"])


def work(case):
    B, rows, page = case["B"], case["gamma"] + 1, case["page"]
    if case["op"] == "plan":
        # both rounds: lengths, tokens and page counts of each sequence, the pages that change hands, slots and positions
        new = B * (rows // page + 1)
        return {"bytes": 2 * (20 * B + 12 * new + 8 * B * rows), "flops": 2 * B * (rows + 8)}
    held = case["D"] + 8                                   # bytes of one token's key and value in the cache
    if case["op"] == "store":
        tokens = B * rows * case["heads"] * (0.5 if case["fused"] else 1.0)
        values = 4 * case["D"]
        return {"bytes": tokens * (2 * values + 2 * held), "flops": tokens * 12 * case["D"]}
    tokens = B * case["heads"] * (case["length"] * (0.75 if B > 1 else 1.0) + rows / 2)
    queries = B * rows * case["group"] * case["heads"] * (0.5 if case["ragged"] else 1.0)
    return {"bytes": tokens * held + queries * 4 * case["D"], "flops": 4 * case["D"] * tokens * rows * case["group"] * (0.5 if case["ragged"] else 1.0)}


# ------------------------------------------------------------------ the definitions in 64 bits

def _exact_rows(x):
    """What the format holds of rows [.., D]; its numbers are rounded where the format rounds them, to 32 bits and to the model's type."""
    d = x.double()
    low, high = d.min(-1, keepdim=True).values, d.max(-1, keepdim=True).values
    step = ((high - low).float().double() / 15).float().to(x.dtype).double()
    share = (1 / step).float().double().nan_to_num(posinf=0.0) * (d - low).float().double()
    return torch.round(share.float().double()).clamp(0, 15) * step + low


def _exact_store(s):
    there = (s["slots"] >= 0)[..., None, None]
    return tuple(torch.where(there, _exact_rows(s[n]), 0.0) for n in ("k", "v"))


def _exact_attend(s):
    case, table, page, D = s["case"], s["table"], s["case"]["page"], s["case"]["D"]
    B, rows, heads, group = case["B"], case["gamma"] + 1, case["heads"], case["group"]
    q = s["q"].double().view(B, rows, heads, group, D)
    out = torch.zeros(B, rows, heads, group, D, dtype=torch.float64, device="cuda")
    lse = torch.zeros(B, rows, heads, group, dtype=torch.float64, device="cuda")
    byte = torch.arange(D, device="cuda") // 2
    shift = torch.arange(D, device="cuda") % 2 * 4
    token = torch.arange(page, device="cuda")
    key_at = token[:, None] * (D // 2) + byte
    unit = torch.arange(D, device="cuda") // 4
    value_at = page * (D // 2) + (token // 2)[:, None] * D + unit * 4 + (token % 2)[:, None] * 2 + byte % 2
    for b in range(B):
        last = rows if s["gamma_b"] is None else int(s["gamma_b"][b]) + 1
        if last < 1:
            continue
        tokens = int(s["lengths"][b]) + last
        ids = table[b, :-(-tokens // page)].long()
        for h in range(heads):
            block = s["cache"][ids, h]
            numbers = block[:, page * D:].contiguous().view(s["q"].dtype).double().view(-1, page, 4)
            k = (((block[:, key_at] >> shift) & 15).double() * numbers[..., 0:1] + numbers[..., 1:2]).flatten(0, 1)[:tokens]
            v = (((block[:, value_at] >> shift) & 15).double() * numbers[..., 2:3] + numbers[..., 3:4]).flatten(0, 1)[:tokens]
            for i in range(last):
                n = int(s["lengths"][b]) + i + 1
                z = q[b, i, h] @ k[:n].T / math.sqrt(D)
                lse[b, i, h] = torch.logsumexp(z, -1)
                out[b, i, h] = torch.softmax(z, -1) @ v[:n]
    out, lse = out.view(s["q"].shape), lse.view(s["q"].shape[:3])
    return (out, lse) if case["lse"] else out


def exact(case, seed):
    if case["op"] == "plan":
        return None                     # whole numbers: nothing is rounded
    state = prepare(case, seed)
    return _exact_store(state) if case["op"] == "store" else _exact_attend(state)
