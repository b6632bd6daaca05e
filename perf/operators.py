"""The operators on logits rows around the verify step, as measured cases.

Three operators work on the rows [.., V] that a round of speculative decoding
has in hand (target rows [B, gamma+1, V], draft rows [B, gamma, V]):

``adjust``   penalties for repeated tokens, biases and grammar masks: what a
             server applies to the rows before the verify step.  Row i of a
             round has the drafts d_0 .. d_{i-1} behind it, so they count as
             generated tokens there.
``top``      the record of a teacher's row that distillation reads: its k best
             log-probabilities, ordered by (logit descending, index ascending),
             and the log of the mass outside them.
``distill``  the loss of a student's (drafter's) row against such a record and
             its gradient: "train" through autograd (forward, then backward),
             "fused" as one call that forms both, "loss" the loss alone.

``run`` computes an operator's plain form from elementary torch operations in
32 bits where ``own`` is false, and calls the package where it is true;
``exact`` computes the definition in 64 bits.
"""

import math

import torch

own = False

_TYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
_BYTES = {"f32": 4, "bf16": 2, "f16": 2}
# a drawn case's rows * V stays below this (the largest listed case of its kind is above it)
_MOST = {"adjust": 3.4e8, "top": 3.4e8, "distill": 5.0e8}


def _package():
    import speculative_decoding_verification_46_gb300 as package

    return package


def _adjust(name, B, gamma, V, dtype, history, penalties, bias, masked, allowed, ragged):
    """history: capacity of a sequence's token history; bias: entries a
    sequence; masked: share of the rows under a grammar; allowed: share of the
    vocabulary a grammar state allows; ragged: drafts differ by sequence."""
    return {"name": name, "op": "adjust", "B": B, "gamma": gamma, "V": V, "dtype": dtype, "history": history, "penalties": penalties,
            "bias": bias, "masked": masked, "allowed": allowed, "ragged": ragged}


def _top(name, rows, V, dtype, k, temperature):
    return {"name": name, "op": "top", "rows": rows, "V": V, "dtype": dtype, "k": k, "temperature": temperature}


def _distill(name, form, rows, V, dtype, k, temperature, tail, ignored):
    """tail: the record carries the mass outside its k tokens; ignored: share
    of the rows with weight zero (padding, prompt positions)."""
    return {"name": name, "op": "distill", "form": form, "rows": rows, "V": V, "dtype": dtype, "k": k, "temperature": temperature,
            "tail": tail, "ignored": ignored}


def listed():
    return [
        # one sequence, one new token, a short chat: the smallest call of a decode loop, all latency
        _adjust("adjust_b1_g0_v32000_bf16", 1, 0, 32000, "bf16", 512, True, 0, 0.0, 1.0, False),
        # a verify round of a medium batch: every request sets penalties and a few biases, a quarter writes under a grammar
        _adjust("adjust_b64_g4_v128256_bf16", 64, 4, 128256, "bf16", 4096, True, 16, 0.25, 0.02, False),
        # an odd vocabulary in half precision, drafts of different lengths, every row under a loose grammar
        _adjust("adjust_b13_g3_v50001_f16_ragged", 13, 3, 50001, "f16", 1500, True, 300, 1.0, 0.6, True),
        # the largest round, after long chats
        _adjust("adjust_b256_g8_v152064_bf16", 256, 8, 152064, "bf16", 8192, True, 16, 0.1, 0.02, False),
        # the record of one small round in single precision
        _top("top_r20_v1024_f32_k8", 20, 1024, "f32", 8, 1.0),
        # a medium round with a wide record
        _top("top_r320_v128256_bf16_k256", 320, 128256, "bf16", 256, 1.0),
        # the record of the largest round, kept while serving
        _top("top_r2304_v152064_bf16_k64", 2304, 152064, "bf16", 64, 0.8),
        # a small drafter's training step on one short round in single precision
        _distill("distill_train_r20_v1024_f32_k8", "train", 20, 1024, "f32", 8, 1.0, True, 0.0),
        # an odd vocabulary in half precision, no tail in the record, a third of the rows padding
        _distill("distill_train_r500_v50001_f16_k33", "train", 500, 50001, "f16", 33, 2.0, False, 0.33),
        # a training step on packed sequences through autograd
        _distill("distill_train_r2048_v128256_bf16_k64", "train", 2048, 128256, "bf16", 64, 1.0, True, 0.1),
        # the same with loss and gradient formed by one call: the largest
        _distill("distill_fused_r4096_v128256_bf16_k64", "fused", 4096, 128256, "bf16", 64, 1.0, True, 0.1),
        # a held-out loss without a gradient
        _distill("distill_loss_r1024_v152064_bf16_k128", "loss", 1024, 152064, "bf16", 128, 1.0, True, 0.0),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["adjust", "top", "distill", "distill"])
    V = _log_int(rng, 1000, 152064)
    if rng.random() < 0.5:
        V = max(8, V // 8 * 8)          # whole 16-byte vectors, as most vocabularies are padded to
    dtype = rng.choice(["bf16", "bf16", "f16", "f32"])
    most = _MOST[op] * 2 / _BYTES[dtype] / V
    if op == "adjust":
        gamma = rng.randint(0, 8)
        B = _log_int(rng, 1, max(1, min(256, int(most / (gamma + 1)))))
        masked, bias = rng.choice([0.0, 0.25, 1.0]), rng.choice([0, 16, 300])
        return _adjust("", B, gamma, V, dtype, _log_int(rng, 16, 8192), rng.random() < 0.8 or not (masked or bias), bias, masked,
                       rng.choice([0.02, 0.6]) if masked else 1.0, rng.random() < 0.3)
    rows = _log_int(rng, 1, max(1, min(4096, int(most))))
    temperature = rng.choice([0.7, 1.0, 2.0])
    if op == "top":
        return _top("", rows, V, dtype, _log_int(rng, 1, 256), temperature)
    k = _log_int(rng, 8, 256)
    return _distill("", rng.choice(["train", "fused", "loss"]), rows, V, dtype, k, temperature, rng.random() < 0.7, rng.choice([0.0, 0.1, 0.33]))


# ------------------------------------------------------------------ inputs

def _heavy_tailed(rows, V, dtype, gen, noise=0.5):
    """Rows like a language model's: logit -1.1 ln(rank) of a random rank plus noise."""
    out = torch.empty(rows, V, dtype=dtype, device="cuda")
    step = max(1, (1 << 28) // V)
    for r in range(0, rows, step):
        n = min(step, rows - r)
        u = torch.rand(n, V, generator=gen, device="cuda").mul_(V).add_(1.0).log_().mul_(-1.1)
        out[r:r + n] = u.add_(torch.randn(n, V, generator=gen, device="cuda"), alpha=noise)
    return out


def _zipf_tokens(shape, V, gen):
    """Token ids whose frequencies fall as text's do."""
    u = torch.rand(shape, generator=gen, device="cuda")
    ranks = torch.exp(u * math.log(V)).long().clamp_(1, V) - 1
    return (ranks * 7919 % V).to(torch.int32)


def _prepare_adjust(case, gen):
    B, gamma, V = case["B"], case["gamma"], case["V"]
    rows = B * (gamma + 1)
    s = {"case": case, "logits": _heavy_tailed(rows, V, _TYPES[case["dtype"]], gen).view(B, gamma + 1, V)}
    s["draft"] = _zipf_tokens((B, gamma), V, gen)
    s["history"] = s["history_len"] = s["prompt_len"] = s["repetition"] = s["frequency"] = s["presence"] = None
    if case["penalties"]:
        H = case["history"]
        s["history"] = _zipf_tokens((B, H), V, gen)
        s["history_len"] = torch.randint(H // 2, H + 1, (B,), generator=gen, device="cuda", dtype=torch.int32)
        s["prompt_len"] = (s["history_len"].float() * torch.rand(B, generator=gen, device="cuda")).to(torch.int32)
        s["repetition"] = 1.0 + 0.3 * torch.rand(B, generator=gen, device="cuda")
        s["frequency"] = 0.5 * torch.rand(B, generator=gen, device="cuda")
        s["presence"] = 0.5 * torch.rand(B, generator=gen, device="cuda")
    s["bias_tokens"] = s["bias_values"] = None
    if case["bias"]:
        n = min(case["bias"], V)
        s["bias_tokens"] = torch.rand(B, V, generator=gen, device="cuda").topk(n, 1).indices.to(torch.int32)
        s["bias_values"] = 4.0 * torch.randn(B, n, generator=gen, device="cuda")
        s["bias_tokens"][:, n - n // 4:] = -1            # requests list fewer than the batch's width
    s["mask"] = s["mask_index"] = None
    if case["masked"]:
        states = 24                                       # the grammar's states that this batch is in
        bits = torch.rand(states, (V + 31) // 32, 32, generator=gen, device="cuda") < case["allowed"]
        bits[:, 0, 0] = True
        words = (bits.long() << torch.arange(32, device="cuda")).sum(-1)
        s["mask"] = torch.where(words >= 1 << 31, words - (1 << 32), words).to(torch.int32)
        index = torch.randint(0, states, (B, gamma + 1), generator=gen, device="cuda", dtype=torch.int32)
        index[torch.rand(B, generator=gen, device="cuda") >= case["masked"]] = -1
        s["mask_index"] = index
    s["gamma_b"] = torch.randint(0, gamma + 1, (B,), generator=gen, device="cuda", dtype=torch.int32) if case["ragged"] else None
    s["out"] = torch.zeros_like(s["logits"])              # the rows behind a ragged sequence's last stay as they are
    return s


def _record(teacher, k, temperature, tail):
    """A teacher's record as it is kept on disk or beside a batch."""
    z = teacher.float() / temperature
    z -= torch.logsumexp(z, -1, keepdim=True)
    best, index = z.topk(k, -1)
    if not tail:
        return index.to(torch.int32), best, None
    return index.to(torch.int32), best, torch.logsumexp(z.scatter_(-1, index, -math.inf), -1)


def _prepare_distill(case, gen):
    rows, V, dtype = case["rows"], case["V"], _TYPES[case["dtype"]]
    s = {"case": case, "student": torch.empty(rows, V, dtype=dtype, device="cuda")}
    s["indices"] = torch.empty(rows, case["k"], dtype=torch.int32, device="cuda")
    s["logprobs"] = torch.empty(rows, case["k"], device="cuda")
    s["tail"] = torch.empty(rows, device="cuda") if case["tail"] else None
    step = max(1, (1 << 27) // V)
    for r in range(0, rows, step):
        n = min(step, rows - r)
        teacher = _heavy_tailed(n, V, dtype, gen)
        s["student"][r:r + n] = teacher + 0.7 * torch.randn(n, V, generator=gen, device="cuda")
        index, best, tail = _record(teacher, case["k"], case["temperature"], case["tail"])
        s["indices"][r:r + n], s["logprobs"][r:r + n] = index, best
        if case["tail"]:
            s["tail"][r:r + n] = tail
    weight = torch.rand(rows, generator=gen, device="cuda") + 0.5
    weight[torch.rand(rows, generator=gen, device="cuda") < case["ignored"]] = 0.0
    # a mean over the rows; half precision trains under a loss scale
    s["weight"] = weight / rows * (2.0 ** 14 if case["dtype"] == "f16" else 1.0)
    if case["form"] == "train":
        s["student"].requires_grad_()
    return s


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    if case["op"] == "adjust":
        return _prepare_adjust(case, gen)
    if case["op"] == "distill":
        return _prepare_distill(case, gen)
    logits = _heavy_tailed(case["rows"], case["V"], _TYPES[case["dtype"]], gen)
    s = {"case": case, "logits": logits}
    # what a server keeps beside the rows: zero-filled scratch, enough for any of these calls
    s["workspace"] = torch.zeros(case["rows"] * 4096 + (64 << 20), dtype=torch.uint8, device="cuda")
    return s


# ------------------------------------------------------------------ the plain forms

def _plain_adjust(s):
    x = s["logits"].float()
    B, rows, V = x.shape
    if s["history"] is not None:
        at = torch.arange(s["history"].shape[1], device=x.device)
        token = s["history"].long()
        zeros = torch.zeros(B, V, device=x.device)
        behind = at >= s["prompt_len"][:, None]
        count = zeros.scatter_add(1, token, (behind & (at < s["history_len"][:, None])).float())
        prompt = zeros.scatter_add(1, token, ((~behind) & (at < s["history_len"][:, None])).float()) > 0
        drafted = torch.zeros(B, rows, V, device=x.device)
        if rows > 1:
            drafted[:, 1:].scatter_(2, s["draft"].long()[:, :, None], 1.0)
        count = count[:, None] + drafted.cumsum(1)
        seen = prompt[:, None] | (count > 0)
        r = s["repetition"][:, None, None]
        x = torch.where(seen, torch.where(x > 0, x / r, x * r), x)
        x = x - s["frequency"][:, None, None] * count - s["presence"][:, None, None] * (count > 0)
    if s["bias_tokens"] is not None:
        listed_ = s["bias_tokens"] >= 0
        bias = torch.zeros(B, V, device=x.device).scatter_add(1, s["bias_tokens"].clamp(min=0).long(), s["bias_values"] * listed_)
        x = x + bias[:, None]
    if s["mask"] is not None:
        v = torch.arange(V, device=x.device)
        allowed = ((s["mask"][:, v // 32] >> (v % 32)) & 1).bool()
        x = torch.where((s["mask_index"] < 0)[..., None] | allowed[s["mask_index"].clamp(min=0).long()], x, -math.inf)
    x = x.to(s["logits"].dtype)
    if s["gamma_b"] is not None:
        x = torch.where((torch.arange(rows, device=x.device) <= s["gamma_b"][:, None])[..., None], x, s["out"])
    return x


def _plain_top(s):
    k, V = s["case"]["k"], s["case"]["V"]
    x = s["logits"].float() + 0.0                          # one zero, whatever its sign
    bits = x.view(torch.int32)
    key = torch.where(bits < 0, ~bits ^ -(1 << 31), bits).long()
    key = (key << 32) + (V - torch.arange(V, device=x.device))       # of equal logits the lowest index is the largest key
    index = key.topk(k, -1).indices
    del key, bits
    top, T = x.amax(-1, keepdim=True), s["case"]["temperature"]
    e = torch.exp((x - top) / T)
    # the few sums and logarithms in 64 bits: a tail of nearly everything has a logarithm next to zero
    total, rest = e.sum(-1, dtype=torch.float64).log(), e.scatter(-1, index, 0.0).sum(-1, dtype=torch.float64).log()
    lp = (x.gather(-1, index) - top).double() / T - total[:, None]
    return index.to(torch.int32), lp.float(), (rest - total).float()


def _plain_distill(s, want_gradient):
    case, T = s["case"], s["case"]["temperature"]
    x, index, w = s["student"].detach().float(), s["indices"].long(), s["weight"]
    top = x.amax(-1, keepdim=True)
    e = torch.exp((x - top) / T)
    # 64 bits for what is summed up and for the few entries of the record: the loss is the small difference of their logarithms
    total = e.sum(-1, keepdim=True, dtype=torch.float64)
    lq = (x.gather(-1, index) - top).double() / T - total.log()
    lp = s["logprobs"].double()
    if case["tail"]:
        rest = e.scatter(-1, index, 0.0).sum(-1, keepdim=True, dtype=torch.float64)
        lp = torch.cat([lp, s["tail"].double()[:, None]], -1)
        lq = torch.cat([lq, rest.log() - total.log()], -1)
    lp = lp - torch.exp(lp).sum(-1, keepdim=True).log()
    p = torch.exp(lp)
    loss = (w * (p * (lp - lq)).sum(-1)).float()
    if not want_gradient:
        return loss
    q = e / total.float()
    g = q * (1.0 - p[:, -1:] / (rest / total)).float() if case["tail"] else q
    g = g.scatter(-1, index, (q.gather(-1, index) - p[:, :case["k"]]).float())
    return loss, (g * (w / T)[:, None]).to(s["student"].dtype)


def run(state):
    case = state["case"]
    if case["op"] == "adjust":
        if not own:
            return _plain_adjust(state)
        return _package().adjust_logits(
            state["logits"], draft=state["draft"], history=state["history"], history_len=state["history_len"], prompt_len=state["prompt_len"],
            repetition=state["repetition"], frequency=state["frequency"], presence=state["presence"], bias_tokens=state["bias_tokens"],
            bias_values=state["bias_values"], mask=state["mask"], mask_index=state["mask_index"], gamma_b=state["gamma_b"], out=state["out"])
    if case["op"] == "top":
        if not own:
            return _plain_top(state)
        return _package().top_logits(state["logits"], case["k"], case["temperature"], workspace=state["workspace"])
    if not own:
        return _plain_distill(state, case["form"] != "loss")
    given = (state["student"], state["indices"], state["logprobs"], state["tail"], case["temperature"])
    if case["form"] == "fused":
        return _package().distill_loss_grad(*given, weight=state["weight"])
    loss = _package().distill_loss(*given, weight=state["weight"])
    if case["form"] == "loss":
        return loss
    (gradient,) = torch.autograd.grad(loss.sum(), state["student"])
    return loss.detach(), gradient


def work(case):
    size, V = _BYTES[case["dtype"]], case["V"]
    if case["op"] == "adjust":
        # every row is written; a logit is read where its row's grammar allows it
        share = 1.0 - case["masked"] * (1.0 - case["allowed"])
        rows = case["B"] * (case["gamma"] / 2 if case["ragged"] else case["gamma"]) + case["B"]
        lists = case["B"] * (3 * case["history"] * case["penalties"] + 8 * case["bias"]) + (3 * V if case["masked"] else 0)
        return {"bytes": rows * V * size * (1 + share) + lists, "flops": rows * V + 6 * rows * case["history"] * case["penalties"]}
    entries = case["rows"] * V
    if case["op"] == "top":
        return {"bytes": entries * size + case["rows"] * (8 * case["k"] + 4), "flops": 5 * entries}
    kept = 1.0 - case["ignored"]
    lists = case["rows"] * (8 * case["k"] + 16)
    if case["form"] == "loss":
        return {"bytes": entries * size * kept + lists, "flops": 4 * entries * kept}
    return {"bytes": entries * size * (1 + kept) + lists, "flops": 8 * entries * kept}


# ------------------------------------------------------------------ the definitions in 64 bits

def _exact_adjust(s):
    B, rows, V = s["logits"].shape
    out = s["out"].double()
    for b in range(B):
        bias = torch.zeros(V, dtype=torch.float64, device="cuda")
        if s["bias_tokens"] is not None:
            use = s["bias_tokens"][b] >= 0
            bias[s["bias_tokens"][b][use].long()] = s["bias_values"][b][use].double()
        made, prompt = torch.zeros(V, dtype=torch.int64, device="cuda"), torch.zeros(V, dtype=torch.bool, device="cuda")
        if s["history"] is not None:
            n0, n1 = int(s["prompt_len"][b]), int(s["history_len"][b])
            prompt[s["history"][b, :n0].long()] = True
            made += torch.bincount(s["history"][b, n0:n1].long(), minlength=V)
        for i in range(rows if s["gamma_b"] is None else int(s["gamma_b"][b]) + 1):
            x = s["logits"][b, i].double()
            if s["history"] is not None:
                if i:
                    made[int(s["draft"][b, i - 1])] += 1
                old = prompt | (made > 0)
                r, f, p = (float(s[n][b]) for n in ("repetition", "frequency", "presence"))
                x = torch.where(old & (x > 0), x / r, torch.where(old, x * r, x)) - made * f - (made > 0) * p
            x = x + bias
            if s["mask"] is not None and int(s["mask_index"][b, i]) >= 0:
                words = s["mask"][int(s["mask_index"][b, i])].long()
                allowed = ((words[:, None] >> torch.arange(32, device="cuda")) & 1).reshape(-1)[:V] == 1
                x[~allowed] = -math.inf
            out[b, i] = x
    return out


def _exact_top(s):
    case, k = s["case"], s["case"]["k"]
    index, lp, tail = [], [], []
    for x in s["logits"].split(max(1, (1 << 25) // case["V"])):
        values, order = torch.sort(x.double(), dim=-1, descending=True, stable=True)
        z = values / case["temperature"]
        lse = torch.logsumexp(z, -1)
        index.append(order[:, :k].to(torch.int32))
        lp.append(z[:, :k] - lse[:, None])
        tail.append(torch.logsumexp(z[:, k:], -1) - lse)
    return torch.cat(index), torch.cat(lp), torch.cat(tail)


def _exact_distill(s):
    case, T, k = s["case"], s["case"]["temperature"], s["case"]["k"]
    losses, gradients = [], []
    n = max(1, (1 << 25) // case["V"])
    for r in range(0, case["rows"], n):
        part = slice(r, r + n)
        index, w = s["indices"][part].long(), s["weight"][part].double()
        target = s["logprobs"][part].double()
        lq = torch.log_softmax(s["student"].detach()[part].double() / T, -1)
        outside = torch.ones_like(lq).scatter_(-1, index, 0.0)
        mine = lq.gather(-1, index)
        if case["tail"]:
            target = torch.cat([target, s["tail"][part].double()[:, None]], -1)
            mine = torch.cat([mine, torch.logsumexp(torch.where(outside > 0, lq, -math.inf), -1)[:, None]], -1)
        target = torch.log_softmax(target, -1)
        losses.append(w * (target.exp() * (target - mine)).sum(-1))
        if case["form"] != "loss":
            g = lq.exp()
            g.scatter_add_(-1, index, -target[:, :k].exp())
            if case["tail"]:
                g -= outside * torch.exp(lq + (target[:, -1:] - mine[:, -1:]))
            gradients.append(g * (w / T)[:, None])
    return torch.cat(losses) if case["form"] == "loss" else (torch.cat(losses), torch.cat(gradients))


def exact(case, seed):
    state = prepare(case, seed)
    if case["op"] == "adjust":
        return _exact_adjust(state)
    return _exact_top(state) if case["op"] == "top" else _exact_distill(state)
